// Softmax cross entropy over a vocabulary with the head product inside, and its gradient:
//     l = X W^T  (T x V, never kept),   loss_t = log sum_v exp(l_tv) - l_ty,
//     dX_t = g_t (sum_v p_tv W_v - W_y),   p = softmax(l);   the head W (V x K, bf16) is frozen.
//
// Everything is taken against the target's own logit: with d_v = l_v - l_y and Z = sum over v != y of exp(d_v),
//     loss = log(1 + Z),   p_y - 1 = -Z / (1 + Z),   p_v = exp(d_v) / (1 + Z),
// so small losses and confident tokens keep their digits, and the weights exp(d_v) of a row need no maximum that
// is known only after the whole vocabulary. Steps, over pieces of the tokens (the weights of one piece, bf16,
// are the only T x V sized buffer, 128 MB at most):
//   vl_target   l_y = X_t . W_y in fp32 on the CUDA cores (the tensor cores' fp32 accumulation truncates: over
//               K = 8192 a logit of 12 came out 1e-4 low), one warp per token; checks and counts the targets;
//   vl_gemm<0>  logits tile by tile on the tensor cores (128 tokens x 256 words, K in steps of 64 through a
//               TMA-filled ring, two accumulators in tensor memory so the epilogue overlaps the next tile);
//               epilogue: exp(d_v) rounded to bf16 (the MMA operand of the gradient; a relative 2^-9 of each
//               weight) and its fp32 sum over the tile's words. Where a tile's largest d exceeds 40 its weights
//               are stored relative to that d (a shift per row and tile), so nothing overflows;
//   vl_finish   one warp per token: adds the tiles' sums in order, loss, the weight -Z of the target, the row's
//               factor g / (1 + Z); brings a row whose tiles have shifts to one shift;
//   vl_gemm<1>  dX = weights x W (contraction over the vocabulary, W as the MN-major operand), times the row's
//               factor in fp32, rounded once to bf16; few tiles are split along the vocabulary into fp32 partial
//               sums that vl_reduce adds in order.
// The tensor pipe bounds it: 2 T V K FLOP for the loss, 4 T V K with the gradient (kept weights, no second
// logits product). All sums are in a fixed order: results are deterministic.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace qnf4 {

constexpr int kVlM = 128, kVlN = 256, kVlK = 64;
constexpr int kVlStages = 4;
constexpr int kVlABytes = kVlM * kVlK * 2, kVlBBytes = kVlN * kVlK * 2;
constexpr int kVlStageBytes = kVlABytes + kVlBBytes;
constexpr int kVlSmemBytes = kVlStages * kVlStageBytes + 256 + 1024;
constexpr int kVlThreads = 6 * 32;
constexpr float kVlMaxShift = 40.0f;      // exp(40) x any vocabulary stays far inside fp32 and bf16
constexpr unsigned kStatusTarget = 4u;

struct VlParams {
  int rows, cols;               // valid rows (tokens of the piece) and columns (words, or features of dX)
  int tiles_m, tiles_n, splits; // a work item is (split, n tile, m tile), m fastest
  int nkb, kb_split;            // contraction blocks of 64, and per split
  const int64_t* target;        // <0>: per row, -1: not in the loss
  const float* ly;              // <0>: target logits
  float2* stats;                // <0>: [n tile][rows] (shift, sum)
  __nv_bfloat16* weights;       // <0>: [rows][pitch], or null (loss only)
  int64_t pitch;
  const float* factor;          // <1>: per row
  __nv_bfloat16* out;           // <1>: [rows][cols], when splits == 1
  float* part;                  // <1>: [split][rows][cols] otherwise
};

template <bool GRAD>
__global__ void __launch_bounds__(kVlThreads, 1)
    vl_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const VlParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = base;
  uint8_t* sB = base + kVlStages * kVlABytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(base + kVlStages * kVlStageBytes);
  uint64_t* empty = full + kVlStages;
  uint64_t* tfull = empty + kVlStages;     // [2]
  uint64_t* tempty = tfull + 2;            // [2]
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t IDESC = idesc_bf16(kVlM, kVlN, false, GRAD);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int num_items = p.tiles_m * p.tiles_n * p.splits;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kVlStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], 4); }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) { tma_prefetch_desc(&tmA); tma_prefetch_desc(&tmB); }
  if (warp == 1) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  int issued = 0;

  auto item = [&](int i, int& m0, int& n0, int& split, int& kb0, int& kb1) {
    m0 = (i % p.tiles_m) * kVlM;
    const int r = i / p.tiles_m;
    n0 = (r % p.tiles_n) * kVlN;
    split = r / p.tiles_n;
    kb0 = split * p.kb_split;
    kb1 = min(p.nkb, kb0 + p.kb_split);
  };

  if (warp == 0) {
    // ------------------------------- TMA producer -------------------------------
    if (lane == 0) {
      int it = 0;
      for (int i = blockIdx.x; i < num_items && !*abort_flag; i += gridDim.x) {
        int m0, n0, split, kb0, kb1;
        item(i, m0, n0, split, kb0, kb1);
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % kVlStages, r = it / kVlStages;
          if (it >= kVlStages && !mbar_wait(&empty[s], (r - 1) & 1)) { *abort_flag = 1; break; }
          if (*abort_flag) break;
          mbar_arrive_expect_tx(&full[s], kVlStageBytes);
          tma_load_2d(sA + s * kVlABytes, &tmA, &full[s], kb * kVlK, m0);
          if constexpr (!GRAD) {
            tma_load_2d(sB + s * kVlBBytes, &tmB, &full[s], kb * kVlK, n0);
          } else {
#pragma unroll
            for (int a = 0; a < kVlN / 64; ++a)
              tma_load_2d(sB + s * kVlBBytes + a * 8192, &tmB, &full[s], n0 + 64 * a, kb * kVlK);
          }
          issued = it + 1;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------- MMA issuer -------------------------------
    if (lane == 0) {
      int it = 0, lt = 0;
      bool ok = true;
      for (int i = blockIdx.x; i < num_items && ok; i += gridDim.x, ++lt) {
        int m0, n0, split, kb0, kb1;
        item(i, m0, n0, split, kb0, kb1);
        const int b = lt & 1, u = lt >> 1;
        if (lt >= 2 && !mbar_wait(&tempty[b], (u - 1) & 1)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(b * kVlN);
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % kVlStages;
          if (!mbar_wait(&full[s], (it / kVlStages) & 1) || *abort_flag) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(sA + s * kVlABytes), b_addr = smem_u32(sB + s * kVlBBytes);
#pragma unroll
          for (int k = 0; k < kVlK / 16; ++k) {
            const uint64_t ad = sdesc_sw128(a_addr + 32u * k, 16u, 1024u);
            const uint64_t bd = GRAD ? sdesc_sw128(b_addr + 2048u * k, 8192u, 1024u)
                                     : sdesc_sw128(b_addr + 32u * k, 16u, 1024u);
            umma_bf16_ss(d, ad, bd, IDESC, (kb > kb0 || k > 0) ? 1u : 0u);
          }
          umma_commit(&empty[s]);
        }
        if (!ok) break;
        umma_commit(&tfull[b]);
      }
      if (!ok) *abort_flag = 1;
      umma_commit(drain);
    }
  } else {
    // ------------------------------- epilogue: one row per thread -------------------------------
    const int q = warp & 3;
    int lt = 0;
    for (int i = blockIdx.x; i < num_items; i += gridDim.x, ++lt) {
      int m0, n0, split, kb0, kb1;
      item(i, m0, n0, split, kb0, kb1);
      const int b = lt & 1, u = lt >> 1;
      const bool ok = mbar_wait(&tfull[b], u & 1);
      if (!__all_sync(0xffffffffu, ok && !*abort_flag)) { *abort_flag = 1; break; }
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(b * kVlN);
      const int row = m0 + 32 * q + lane;
      const bool live = row < p.rows;
      const int ncol = min(kVlN, p.cols - n0);
      if constexpr (!GRAD) {
        const float ly = live ? p.ly[row] : 0.0f;
        const int64_t yt = live ? p.target[row] - n0 : -1;
        const int y = (yt >= 0 && yt < ncol) ? static_cast<int>(yt) : -1;   // the target's column, if it is here
        // the largest d; a NaN is kept (it makes the row's sum NaN), the target's own column is left out
        float top = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < ncol; c += 16) {
          uint32_t v[16];
          tmem_ld16(taddr + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float l = __uint_as_float(v[j]);
            if (c + j < ncol && c + j != y) top = fmaxf(top, l);
          }
        }
        const float shift = top - ly > kVlMaxShift ? top - ly : 0.0f;
        const float ref = ly + shift;
        float sum = 0.0f;
#pragma unroll 1
        for (int c = 0; c < ncol; c += 16) {
          uint32_t v[16];
          tmem_ld16(taddr + c, v);
          tmem_wait_ld();
          uint32_t o[8];
          float e[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float w = __expf(__uint_as_float(v[j]) - ref);
            e[j] = (c + j < ncol && c + j != y) ? w : 0.0f;
          }
          float part = 0.0f;
#pragma unroll
          for (int j = 0; j < 16; ++j) part += e[j];
          sum += part;
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = pack_bf16x2(e[2 * j], e[2 * j + 1]);
          if (p.weights && live) {               // the pitch has room up to a multiple of 16 words
            uint4* dst = reinterpret_cast<uint4*>(p.weights + row * p.pitch + n0 + c);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
          }
          __syncwarp();                          // the next tcgen05.ld is warp-wide
        }
        if (live) p.stats[static_cast<int64_t>(n0 / kVlN) * p.rows + row] = make_float2(shift, sum);
      } else {
        const float f = p.splits == 1 && live ? p.factor[row] : 0.0f;
#pragma unroll 1
        for (int c = 0; c < ncol; c += 16) {
          uint32_t v[16];
          tmem_ld16(taddr + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < 2; ++h) {          // K % 8 == 0: whole groups of 8
            if (!live || c + 8 * h >= ncol) break;
            if (p.splits == 1) {
              uint32_t o[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float lo = __uint_as_float(v[8 * h + 2 * j]), hi = __uint_as_float(v[8 * h + 2 * j + 1]);
                o[j] = f != 0.0f ? pack_bf16x2(lo * f, hi * f) : 0u;
              }
              *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(row) * p.cols + n0 + c + 8 * h) =
                  make_uint4(o[0], o[1], o[2], o[3]);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(
                  p.part + (static_cast<int64_t>(split) * p.rows + row) * p.cols + n0 + c + 8 * h);
              dst[0] = make_uint4(v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3]);
              dst[1] = make_uint4(v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]);
            }
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[b]);
    }
  }

  // ------------------------------- teardown -------------------------------
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if (warp == 0 && lane == 0)
      for (int it = (issued > kVlStages ? issued - kVlStages : 0); it < issued; ++it)
        mbar_wait_short(&full[it % kVlStages], (it / kVlStages) & 1);
    if (warp == 1 && lane == 0) mbar_wait_short(drain, 0);
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// One warp per token: the target (-1 where the token takes no part; a target outside the vocabulary is
// reported in the status word and left out too), its logit in fp32, and the count of tokens in the loss.
template <typename TI>
__global__ void __launch_bounds__(256) vl_target_kernel(const __nv_bfloat16* __restrict__ X,
                                                        const __nv_bfloat16* __restrict__ W,
                                                        const TI* __restrict__ targets, int64_t T, int64_t V, int K,
                                                        int64_t ignore, int64_t* __restrict__ target,
                                                        float* __restrict__ ly, unsigned long long* count) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  if (t >= T) return;
  const int64_t y = static_cast<int64_t>(targets[t]);
  const bool in = y != ignore && y >= 0 && y < V;
  if (!in) {
    if (lane == 0) {
      if (y != ignore) raise_status(kStatusTarget);
      target[t] = -1;
      ly[t] = 0.0f;
    }
    return;
  }
  const uint4* x = reinterpret_cast<const uint4*>(X + t * K);
  const uint4* w = reinterpret_cast<const uint4*>(W + y * K);
  float acc = 0.0f;
  for (int i = lane; i < K / 8; i += 32) {
    const uint4 a = x[i], b = w[i];
    const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {     // a bf16 is the upper half of its fp32
      s = fmaf(__uint_as_float(av[j] << 16), __uint_as_float(bv[j] << 16), s);
      s = fmaf(__uint_as_float(av[j] & 0xffff0000u), __uint_as_float(bv[j] & 0xffff0000u), s);
    }
    acc += s;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) {
    target[t] = y;
    ly[t] = acc;
    atomicAdd(count, 1ull);           // an integer: the order does not matter
  }
}

// One warp per token of the piece.
__global__ void __launch_bounds__(256) vl_finish_kernel(const float2* __restrict__ stats, int rows, int tiles,
                                                        const int64_t* __restrict__ target, int V,
                                                        const float* __restrict__ dloss, int mean,
                                                        const unsigned long long* __restrict__ count,
                                                        float* __restrict__ loss, __nv_bfloat16* weights,
                                                        int64_t pitch, float* __restrict__ factor) {
  const int lane = threadIdx.x & 31;
  const int row = static_cast<int>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  if (row >= rows) return;
  const int64_t y = target[row];
  if (y < 0) {
    if (lane == 0) {
      loss[row] = 0.0f;
      if (factor) factor[row] = 0.0f;
    }
    return;
  }
  float shift = 0.0f;                 // the row's: the largest of its tiles'
  for (int i = lane; i < tiles; i += 32) shift = fmaxf(shift, stats[static_cast<int64_t>(i) * rows + row].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) shift = fmaxf(shift, __shfl_xor_sync(0xffffffffu, shift, o));
  float z = 0.0f;
  for (int i = lane; i < tiles; i += 32) {
    const float2 s = stats[static_cast<int64_t>(i) * rows + row];
    z += shift > 0.0f ? s.y * expf(s.x - shift) : s.y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  const float one = shift > 0.0f ? expf(-shift) : 1.0f;
  if (lane == 0) loss[row] = shift > 0.0f ? shift + logf(z + one) : log1pf(z);
  if (!weights) return;
  __nv_bfloat16* w = weights + static_cast<int64_t>(row) * pitch;
  if (shift > 0.0f) {
    for (int v = lane; v < V; v += 32) {
      const float s = stats[static_cast<int64_t>(v / kVlN) * rows + row].x;
      if (s != shift) w[v] = __float2bfloat16_rn(__bfloat162float(w[v]) * expf(s - shift));
    }
    __syncwarp();
  }
  if (lane == 0) {
    w[y] = __float2bfloat16_rn(-z);
    float g = dloss ? dloss[row] : 1.0f;
    if (mean) g /= static_cast<float>(*count);
    factor[row] = g / (z + one);
  }
}

// dX from the partial sums of the vocabulary's splits, in order.
__global__ void __launch_bounds__(256) vl_reduce_kernel(const float4* __restrict__ part, int splits, int64_t rows,
                                                        int64_t cols4, const float* __restrict__ factor,
                                                        uint2* __restrict__ out) {
  const int64_t n = rows * cols4;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    float4 a = part[i];
    for (int s = 1; s < splits; ++s) {
      const float4 b = part[s * n + i];
      a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
    }
    const float f = factor[i / cols4];
    out[i] = f != 0.0f ? make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f)) : make_uint2(0u, 0u);
  }
}

// total = sum of the tokens' losses (fp64, fixed order), over their count for a mean (0 / 0 = NaN when no
// token is in the loss).
__global__ void __launch_bounds__(1024) vl_total_kernel(const float* __restrict__ loss, int64_t T, int mean,
                                                        const unsigned long long* __restrict__ count,
                                                        float* __restrict__ total) {
  __shared__ double sm[32];
  double a = 0.0;
  for (int64_t i = threadIdx.x; i < T; i += blockDim.x) a += loss[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x < 32) {
    a = sm[threadIdx.x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (threadIdx.x == 0) *total = static_cast<float>(mean ? a / static_cast<double>(*count) : a);
  }
}

}  // namespace qnf4
