// Rotary positions: every pair (a, b) of the first rotary_dim features of a head is turned by the angle
// p * theta_i of its token's position p, and scaled by m:
//     a' = m (a cos - b sin),   b' = m (b cos + a sin);
// the pairs are features (i, i + R/2) (half layout) or (2i, 2i + 1) (interleaved). The rest of the head
// passes through. The gradient of a rotation is the rotation by -p theta, so `inverse` is the backward.
//
// What bounds it: HBM, one read and one write of every element (3 FLOP per element). The angles are shared
// by all heads of a token: a CTA of 128 threads first forms the sines and cosines of its 2 tokens (of one batch
// row) in shared memory, one per thread, and then every thread keeps one chunk of pairs and walks over the heads of
// both tensors, the tokens' 16-byte accesses (where sizes and strides allow them) in flight together before any is
// turned and stored: the compiler may not move a load over a store that could be in place. Neighbouring slots of a
// CTA are neighbouring heads, whose features are one run of memory. Measured for 8192 tokens of 64 heads of 128
// features (268 MB, 41 us at the copy's rate): 46 us, 5.9 TB/s; with 256 threads 52, 512 threads 85 (larger CTAs
// wait longer for their set-up), 1 / 4 tokens per CTA 50 / 58, slots that are tokens 170 (256-byte pieces 24 KB
// apart).
//
// Angles: p * theta / (2 pi) is formed in fp64, where even p = 2^31 leaves 2^-22 of a turn; its fraction of a
// turn, in [-1/2, 1/2], is rounded once to fp32 and goes to sincospif. Everything else is fp32, rounded once
// to the element type at the end.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace qnf4 {

constexpr int kRopeMaxPairs = 256;     // rotary_dim <= 512
constexpr int kRopeThreads = 128;      // units of one head x head slots, at most (more only when one head has more)
constexpr int kRopeMaxTensors = 2;
constexpr int kRopeTokens = 2;          // tokens per CTA, where there are many

struct RopeSide {                      // one tensor: heads x head_dim per token; strides in elements
  const void* in;
  void* out;
  int64_t in_b, in_t, in_h, out_b, out_t, out_h;
};
struct RopeParams {
  RopeSide x[kRopeMaxTensors];
  int heads0, heads;                   // heads of x[0], and of all tensors together
  int64_t B, T;                        // batch rows, tokens per row
  int rotary_dim, head_dim;
  int units, tail, tail_aligned;       // chunks of pairs per head, and 16-byte chunks copied per head
  int slots;                           // heads that one CTA works on at a time
  int heads_per_cta;
  const void* positions;               // null: the token's index within its row
  int pos64;
  int64_t pos_b, offset;
  float mscale;
  int inverse;
  double turns[kRopeMaxPairs];         // theta_i / (2 pi)
};

template <typename T> __device__ __forceinline__ float rope_load(T v);
template <> __device__ __forceinline__ float rope_load(float v) { return v; }
template <> __device__ __forceinline__ float rope_load(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T rope_store(float v);
template <> __device__ __forceinline__ float rope_store(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 rope_store(float v) { return __float2bfloat16_rn(v); }

template <typename T, int VE, int AL>
struct alignas(sizeof(T) * AL) RopeVec { T v[VE]; };

// Results are written once and not read here: 16-byte stores stream past L2's resident lines (49 to 46 us for 8192
// tokens of 64 heads).
template <typename V> __device__ __forceinline__ void rope_put(V* p, const V& v) {
  if constexpr (sizeof(V) == 16) __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&v));
  else *p = v;
}
// Cosine and sine of one pair at token t of row b, times the scale.
__device__ __forceinline__ void rope_angle(const RopeParams& p, int64_t b, int64_t t, int pair, float& cosine, float& sine) {
  int64_t pos = t;
  if (p.positions) {
    const int64_t at = b * p.pos_b + t;
    pos = p.pos64 ? static_cast<const int64_t*>(p.positions)[at]
                  : static_cast<int64_t>(static_cast<const int32_t*>(p.positions)[at]);
  }
  pos += p.offset;
  const double turn = static_cast<double>(pos) * p.turns[pair];
  const float frac = static_cast<float>(turn - rint(turn));
  float s, c;
  sincospif(2.0f * frac, &s, &c);
  cosine = c * p.mscale;
  sine = (p.inverse ? -s : s) * p.mscale;
}

// VE: elements of one access, aligned to AL elements (AL < VE only for interleaved pairs at odd strides). Half
// layout: a unit is VE features of the first half and the VE that pair with them; interleaved: VE / 2 pairs side
// by side. TOK: tokens per CTA.
template <typename T, int VE, int AL, bool HALF, int TOK>
__global__ void rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int PAIRS = HALF ? VE : VE / 2, TAIL = 16 / sizeof(T);
  using Vec = RopeVec<T, VE, AL>;
  extern __shared__ __align__(16) float rope_sm[];   // [cosines, sines][TOK][R/2]
  const int half = p.rotary_dim / 2;
  const float *cs = rope_sm, *sn = rope_sm + TOK * half;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * TOK;
  const int ntok = static_cast<int>(min(static_cast<int64_t>(TOK), p.T - t0));
  const int per_head = p.units + p.tail;
  const int u = threadIdx.x % per_head, slot = threadIdx.x / per_head;
  const int h_end = min(p.heads, static_cast<int>(blockIdx.y + 1) * p.heads_per_cta);
  const bool turned = u < p.units;
  const int f = turned ? u * VE : p.rotary_dim + (u - p.units) * TAIL;

  for (int64_t b = blockIdx.z; b < p.B; b += gridDim.z) {
    for (int e = threadIdx.x; e < ntok * half; e += blockDim.x) {
      const int i = e / half, pair = e - i * half;
      rope_angle(p, b, t0 + i, pair, rope_sm[e], rope_sm[TOK * half + e]);
    }
    __syncthreads();
    for (int h = blockIdx.y * p.heads_per_cta + slot; h < h_end; h += p.slots) {
      const bool second = h >= p.heads0;
      const RopeSide& x = p.x[second ? 1 : 0];
      const int hh = second ? h - p.heads0 : h;
      const int64_t in_t = x.in_t, out_t = x.out_t;
      const T* in = static_cast<const T*>(x.in) + b * x.in_b + t0 * in_t + hh * x.in_h + f;
      T* out = static_cast<T*>(x.out) + b * x.out_b + t0 * out_t + hh * x.out_h + f;
      if (turned) {
        Vec v[TOK][HALF ? 2 : 1];
#pragma unroll
        for (int i = 0; i < TOK; ++i)
          if (i < ntok) {
            v[i][0] = *reinterpret_cast<const Vec*>(in + i * in_t);
            if constexpr (HALF) v[i][1] = *reinterpret_cast<const Vec*>(in + i * in_t + half);
          }
#pragma unroll
        for (int i = 0; i < TOK; ++i)
          if (i < ntok) {
            const float *c = cs + i * half + u * PAIRS, *s = sn + i * half + u * PAIRS;
#pragma unroll
            for (int k = 0; k < PAIRS; ++k) {
              T& va = HALF ? v[i][0].v[k] : v[i][0].v[2 * k];
              T& vb = HALF ? v[i][HALF ? 1 : 0].v[k] : v[i][0].v[2 * k + (HALF ? 0 : 1)];
              const float xa = rope_load(va), xb = rope_load(vb);
              va = rope_store<T>(xa * c[k] - xb * s[k]);
              vb = rope_store<T>(xb * c[k] + xa * s[k]);
            }
            rope_put(reinterpret_cast<Vec*>(out + i * out_t), v[i][0]);
            if constexpr (HALF) rope_put(reinterpret_cast<Vec*>(out + i * out_t + half), v[i][1]);
          }
      } else {                                       // 16 bytes of the features behind the rotated part
        const int n = min(TAIL, p.head_dim - f);
        if (p.tail_aligned && n == TAIL) {
          uint4 v[TOK];
#pragma unroll
          for (int i = 0; i < TOK; ++i)
            if (i < ntok) v[i] = *reinterpret_cast<const uint4*>(in + i * in_t);
#pragma unroll
          for (int i = 0; i < TOK; ++i)
            if (i < ntok) *reinterpret_cast<uint4*>(out + i * out_t) = v[i];
        } else {
          for (int i = 0; i < ntok; ++i)
            for (int k = 0; k < n; ++k) out[i * out_t + k] = in[i * in_t + k];
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace qnf4
