// Y = X W^T for a few tokens (T <= 64) and a 4-bit weight with one fp32 constant per block of 64:
//     W[n][k] = level[code[n][k]] * absmax[n][k / 64],   any codebook of up to 16 levels.
//
// HBM bounds it at a few tokens: 0.5625 B per weight, read once. The contraction runs on mma.sync m16n8k16 (the
// weight as the 16-row A operand, X as the 8-token B operand; a 128-row tensor-memory tile would be padding at
// these token counts). One shared-memory load turns a code byte into the bf16 pair (level[high], level[low]):
// a 256-entry table, one copy per lane so the lookups have no bank conflicts. Inside a block of 64 the MMA's k
// index is permuted alike on both operands, so lane j of a quad holds elements 16 j .. 16 j + 15: 8 code bytes and
// 32 bytes of X in a row. The block's constant multiplies the fp32 result of its four MMAs, so the only rounding
// of a weight is its level's to bf16 (a relative 2^-9), as in the T <= 16 forward of the double-quantized layer.
// The warps of a CTA share a tile of 16 rows and split the contraction; their fp32 sums meet in shared memory and
// are added in warp order, so results are deterministic.
#pragma once

#include "codec.cuh"
#include "common.cuh"
#include "decode_nf4.cuh"

namespace qnf4 {

constexpr int kClWarps = 16;
constexpr int kClMaxTokens = 64;
constexpr int kClTableBytes = 256 * 32 * 4;

struct ClParams {
  int T, N, nkb, tiles;
  const __nv_bfloat16* X;
  const uint8_t* codes;
  const float* absmax;
  __nv_bfloat16* Y;
};

template <int NT>   // token tiles of 8
__global__ void __launch_bounds__(kClWarps * 32, 1) codebook_linear_kernel(const ClParams p, const CodebookArg cb) {
  extern __shared__ __align__(16) uint8_t cl_smem[];
  uint32_t* table = reinterpret_cast<uint32_t*>(cl_smem);
  float* red = reinterpret_cast<float*>(cl_smem + kClTableBytes);   // [warp][16 rows][8 NT tokens]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, j = lane & 3;
  for (int i = threadIdx.x; i < 256 * 32; i += blockDim.x)
    table[i] = pack_bf16x2(cb.levels[i >> 9], cb.levels[(i >> 5) & 15]);
  __syncthreads();
  const uint32_t tab = smem_u32(table) + 4u * lane;
  const int K = p.nkb * 64;

  for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const int64_t r0 = min(tile * 16 + g, p.N - 1), r1 = min(tile * 16 + g + 8, p.N - 1);
    const uint8_t* c0 = p.codes + r0 * (K / 2) + 8 * j;
    const uint8_t* c1 = p.codes + r1 * (K / 2) + 8 * j;
    const float* a0 = p.absmax + r0 * p.nkb;
    const float* a1 = p.absmax + r1 * p.nkb;
    float acc[NT][4] = {};
#pragma unroll 4
    for (int kb = warp; kb < p.nkb; kb += kClWarps) {
      const uint2 w0 = *reinterpret_cast<const uint2*>(c0 + 32 * kb), w1 = *reinterpret_cast<const uint2*>(c1 + 32 * kb);
      const float s0 = a0[kb], s1 = a1[kb];
      uint32_t a[16];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint32_t x0 = (s < 2 ? w0.x : w0.y) >> (16 * (s & 1)), x1 = (s < 2 ? w1.x : w1.y) >> (16 * (s & 1));
        a[4 * s] = dc_lut(tab + ((x0 & 255u) << 7));
        a[4 * s + 1] = dc_lut(tab + ((x1 & 255u) << 7));
        a[4 * s + 2] = dc_lut(tab + (((x0 >> 8) & 255u) << 7));
        a[4 * s + 3] = dc_lut(tab + (((x1 >> 8) & 255u) << 7));
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (8 * n + g < p.T) {
          const uint4* xp = reinterpret_cast<const uint4*>(p.X + static_cast<int64_t>(8 * n + g) * K + 64 * kb + 16 * j);
          x[0] = __ldg(xp);
          x[1] = __ldg(xp + 1);
        }
        float d[4] = {};
#pragma unroll
        for (int s = 0; s < 4; ++s)
          dc_mma(d[0], d[1], d[2], d[3], a[4 * s], a[4 * s + 1], a[4 * s + 2], a[4 * s + 3], dc_word(x[s >> 1], 2 * (s & 1)),
                 dc_word(x[s >> 1], 2 * (s & 1) + 1));
        acc[n][0] = fmaf(s0, d[0], acc[n][0]);
        acc[n][1] = fmaf(s0, d[1], acc[n][1]);
        acc[n][2] = fmaf(s1, d[2], acc[n][2]);
        acc[n][3] = fmaf(s1, d[3], acc[n][3]);
      }
    }
    float* mine = red + warp * 16 * 8 * NT;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mine[g * 8 * NT + 8 * n + 2 * j] = acc[n][0];
      mine[g * 8 * NT + 8 * n + 2 * j + 1] = acc[n][1];
      mine[(g + 8) * 8 * NT + 8 * n + 2 * j] = acc[n][2];
      mine[(g + 8) * 8 * NT + 8 * n + 2 * j + 1] = acc[n][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * 8 * NT; i += blockDim.x) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kClWarps; ++w) sum += red[w * 16 * 8 * NT + i];
      const int n = tile * 16 + i / (8 * NT), t = i % (8 * NT);
      if (n < p.N && t < p.T) p.Y[static_cast<int64_t>(t) * p.N + n] = __float2bfloat16_rn(sum);
    }
    __syncthreads();
  }
}

}  // namespace qnf4
