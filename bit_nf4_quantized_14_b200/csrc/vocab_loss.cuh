// Softmax cross entropy over a vocabulary with the head product inside, and its gradient:
//     l = X W^T  (T x V, never kept),   loss_t = log sum_v exp(l_tv) - l_ty,
//     dX_t = g_t (sum_v p_tv W_v - W_y),   p = softmax(l);   the head W (V x K, bf16) is frozen.
//
// Everything is taken against the target's own logit: with d_v = l_v - l_y and Z = sum over v != y of exp(d_v),
//     loss = log(1 + Z),   p_y - 1 = -Z / (1 + Z),   p_v = exp(d_v) / (1 + Z),
// so small losses and confident tokens keep their digits, and the weights exp(d_v) of a row need no maximum that
// is known only after the whole vocabulary. Tokens whose target is ignored cost nothing: the others are numbered
// first, and the steps run over those rows, in pieces (the weights of one piece, bf16, are the only T x V sized
// buffer, 128 MB at most; the host launches for every token, the kernels read the count and stop at it):
//   vl_index    numbers the tokens in the loss, in order; checks the targets;
//   vl_target   l_y = X_t . W_y in fp32 on the CUDA cores (the tensor cores' fp32 accumulation truncates: over
//               K = 8192 a logit of 12 came out 1e-4 low), one warp per row; copies the rows together where
//               tokens are left out, and zeroes those tokens' gradients;
//   vl_gemm<0>  logits tile by tile on the tensor cores (a CTA pair: 256 rows x up to 256 words, K in steps of 64
//               through a TMA-filled ring, two accumulators in tensor memory so the epilogue overlaps the next tile);
//               epilogue: exp(d_v) rounded to bf16 (the MMA operand of the gradient; a relative 2^-8 of each weight
//               at most) and its fp32 sum over the tile's words. Where a tile's largest d exceeds 40 its weights
//               are stored relative to that d (a shift per row and tile), so nothing overflows;
//   vl_finish   one warp per row: adds the tiles' sums in order, loss, the weight -Z of the target, the row's
//               factor g / (1 + Z); brings a row whose tiles have shifts to one shift;
//   vl_gemm<1>  dX = weights x W (contraction over the vocabulary, W as the MN-major operand), times the row's
//               factor in fp32, rounded once to bf16. Whole waves of tiles run in step along the vocabulary, so W
//               and the weights pass through L2 once; the tiles of a last, partly filled wave are cut along the
//               vocabulary to fill the CTA pairs (2048 x 4096 outputs are 128 tiles for 74 pairs) and leave fp32
//               partial sums that vl_reduce adds in order. (One run of all tiles' steps cut evenly over the pairs
//               filled them too, but every pair read another part of W: 487 against 428 us uncut.)
// The tensor pipe bounds it: 2 T V K FLOP for the loss, 4 T V K with the gradient (kept weights, no second
// logits product). All sums are in a fixed order: results are deterministic.
//
// A CTA pair (tcgen05 cta_group::2) holds half of the rows each and half of the words each in its shared memory, so
// an operand byte is read from shared memory for twice the FLOP; a single CTA takes up to 128 rows (PAIR false),
// where a pair would leave half of its rows empty.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace qnf4 {

constexpr int kVlM = 128, kVlN = 256, kVlK = 64;      // rows per CTA; widest tile; contraction step
constexpr int kVlABytes = kVlM * kVlK * 2;
template <bool PAIR> struct VlCfg {
  static constexpr int CTAS = PAIR ? 2 : 1;
  static constexpr int BROWS = kVlN / CTAS;           // words (or features) of a tile in one CTA's shared memory
  static constexpr int B_BYTES = BROWS * kVlK * 2;
  static constexpr int STAGE_BYTES = kVlABytes + B_BYTES;
  static constexpr int STAGES = PAIR ? 6 : 4;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 256 + 1024;
  static_assert(SMEM_BYTES <= 227 * 1024 && (2 * STAGES + 5) * 8 + 8 <= 256, "shared memory per CTA");
};
constexpr int kVlThreads = 6 * 32;
constexpr float kVlMaxShift = 40.0f;      // exp(40) x any vocabulary stays far inside fp32 and bf16
constexpr unsigned kStatusTarget = 4u;

struct VlParams {
  const int* count;             // tokens in the loss
  int r0, rows_max;             // this piece: rows r0 .. of them, rows_max at most
  int copied;                   // <0>: rows live in the packed copy (second map) when count < copied
  int cols, bn;                 // columns (words, or features of dX) and columns per tile
  int tiles_n, nkb;             // column tiles; contraction blocks of 64
  const int* target;            // <0>: per row
  const float* ly;              // <0>: target logits
  float2* stats;                // <0>: [column tile][rows_max] (shift, sum)
  __nv_bfloat16* weights;       // <0>: [rows][pitch], or null (loss only)
  int64_t pitch;
  const int* token;             // <1>: the token of each row
  const float* factor;          // <1>: per row
  __nv_bfloat16* out;           // <1>: [token][cols]
  float* part;                  // <1>: partial tiles of [128 CTAS][256]
};
__device__ __forceinline__ int vl_rows(const int* count, int r0, int rows_max) {
  return max(0, min(rows_max, *count - r0));
}
// How the gradient's tiles are dealt to its workers: `full` whole ones in full waves, then the others in `cuts`
// parts of the contraction each. The number of cuts minimises what the last wave takes, counted in contraction
// steps, a part's write and read of its fp32 tile as a quarter of a step; at most kVlParts parts per worker.
constexpr int kVlParts = 3;
struct VlDeal { int full, rest, cuts; };
__host__ __device__ __forceinline__ VlDeal vl_deal(int tiles, int workers, int nkb) {
  VlDeal d;
  d.full = tiles / workers * workers;
  d.rest = tiles - d.full;
  d.cuts = 1;
  float best = 1e30f;
  for (int s = 1; s <= 32 && d.rest * s <= kVlParts * workers && s * 4 <= nkb + 3; ++s) {
    const int waves = (d.rest * s + workers - 1) / workers;
    const float cost = static_cast<float>(waves) * nkb / s + (s > 1 ? 0.25f * d.rest * s : 0.0f);
    if (cost < best) { best = cost; d.cuts = s; }
  }
  return d;
}

__device__ __forceinline__ uint32_t vl_peer(uint32_t addr, uint32_t rank) {    // the same address in CTA `rank` of the pair
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
template <bool PAIR>
__device__ __forceinline__ void vl_tma(void* dst, const void* map, uint32_t bar, int c0, int c1) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)), "l"(map), "r"(bar), "r"(c0), "r"(c1) : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            smem_u32(dst)), "l"(map), "r"(bar), "r"(c0), "r"(c1) : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void vl_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    umma_bf16_ss(d, a, b, idesc, accumulate);
}
// Arrive on a barrier (in both CTAs of a pair) once every MMA issued so far by this thread has completed.
template <bool PAIR>
__device__ __forceinline__ void vl_commit(uint64_t* bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)), "h"(static_cast<uint16_t>(3)) : "memory");
  else
    umma_commit(bar);
}
__device__ __forceinline__ void vl_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <bool GRAD, bool PAIR>
__device__ __forceinline__ void vl_gemm(const CUtensorMap& tmA, const CUtensorMap& tmA2, const CUtensorMap& tmB,
                                        const VlParams& p) {
  using C = VlCfg<PAIR>;
  constexpr int ST = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  // 1 KB alignment of the shared address (the same in both CTAs of a pair)
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sA = base;
  uint8_t* sB = base + ST * kVlABytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(base + ST * C::STAGE_BYTES);
  uint64_t* empty = full + ST;
  uint64_t* tfull = empty + ST;            // [2]
  uint64_t* tempty = tfull + 2;            // [2]
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? blockIdx.x & 1 : 0;
  const int worker = PAIR ? blockIdx.x >> 1 : blockIdx.x, workers = PAIR ? gridDim.x >> 1 : gridDim.x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], 4 * C::CTAS); }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) { tma_prefetch_desc(&tmA); tma_prefetch_desc(&tmB); }
  if (warp == 1) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(tmem_slot, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) vl_cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t idesc = idesc_bf16(kVlM * C::CTAS, 16, false, GRAD) - (2u << 17) + (static_cast<uint32_t>(p.bn >> 3) << 17);
  int issued = 0;

  const int rows = vl_rows(p.count, p.r0, p.rows_max);
  const int tiles_m = (rows + kVlM * C::CTAS - 1) / (kVlM * C::CTAS);
  const int tiles = tiles_m * p.tiles_n;
  const VlDeal deal = GRAD ? vl_deal(tiles, workers, p.nkb) : VlDeal{tiles, 0, 1};
  const int num_items = deal.full + deal.rest * deal.cuts;
  const int bn_cta = p.bn / C::CTAS;
  struct Item { int m0, n0, kb0, kb1; };
  auto item = [&](int i) {
    Item t;
    int tile = i;
    t.kb0 = 0;
    t.kb1 = p.nkb;
    if (GRAD && i >= deal.full) {
      const int cut = (i - deal.full) / deal.rest;
      tile = deal.full + (i - deal.full) % deal.rest;
      t.kb0 = static_cast<int>(static_cast<int64_t>(p.nkb) * cut / deal.cuts);
      t.kb1 = static_cast<int>(static_cast<int64_t>(p.nkb) * (cut + 1) / deal.cuts);
    }
    t.m0 = (tile % tiles_m) * kVlM * C::CTAS;
    t.n0 = (tile / tiles_m) * p.bn;
    return t;
  };

  if (warp == 0) {
    // ------------------------------- TMA producer (both CTAs) -------------------------------
    if (lane == 0) {
      const CUtensorMap* ma = !GRAD && *p.count < p.copied ? &tmA2 : &tmA;
      int it = 0;
      for (int i = worker; i < num_items && !*abort_flag; i += workers) {
        const Item t = item(i);
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
          const int s = it % ST, r = it / ST;
          if (it >= ST && !mbar_wait(&empty[s], (r - 1) & 1)) { *abort_flag = 1; break; }
          if (*abort_flag) break;
          // both CTAs' copies complete on the first one's barrier
          const uint32_t bar = PAIR ? vl_peer(smem_u32(&full[s]), 0) : smem_u32(&full[s]);
          if (rank == 0)
            mbar_arrive_expect_tx(&full[s], C::CTAS * (kVlABytes + (GRAD ? C::B_BYTES : bn_cta * kVlK * 2)));
          vl_tma<PAIR>(sA + s * kVlABytes, ma, bar, kb * kVlK, t.m0 + rank * kVlM);
          if constexpr (!GRAD) {
            vl_tma<PAIR>(sB + s * C::B_BYTES, &tmB, bar, kb * kVlK, t.n0 + rank * bn_cta);
          } else {
#pragma unroll
            for (int a = 0; a < C::BROWS / 64; ++a)
              vl_tma<PAIR>(sB + s * C::B_BYTES + a * 8192, &tmB, bar, t.n0 + rank * C::BROWS + 64 * a, kb * kVlK);
          }
          issued = it + 1;
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------- MMA issuer (the first CTA) -------------------------------
    if (lane == 0 && rank == 0) {
      int it = 0, lt = 0;
      bool ok = true;
      for (int i = worker; i < num_items && ok; i += workers, ++lt) {
        const Item t = item(i);
        const int b = lt & 1, u = lt >> 1;
        if (lt >= 2 && !mbar_wait(&tempty[b], (u - 1) & 1)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(b * kVlN);
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
          const int s = it % ST;
          if (!mbar_wait(&full[s], (it / ST) & 1) || *abort_flag) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(sA + s * kVlABytes), b_addr = smem_u32(sB + s * C::B_BYTES);
#pragma unroll
          for (int k = 0; k < kVlK / 16; ++k) {
            const uint64_t ad = sdesc_sw128(a_addr + 32u * k, 16u, 1024u);
            const uint64_t bd = GRAD ? sdesc_sw128(b_addr + 2048u * k, 8192u, 1024u)
                                     : sdesc_sw128(b_addr + 32u * k, 16u, 1024u);
            vl_mma<PAIR>(d, ad, bd, idesc, (kb > t.kb0 || k > 0) ? 1u : 0u);
          }
          vl_commit<PAIR>(&empty[s]);
        }
        if (!ok) break;
        vl_commit<PAIR>(&tfull[b]);
      }
      if (!ok) *abort_flag = 1;
      vl_commit<PAIR>(drain);
    }
  } else {
    // ------------------------------- epilogue: one row per thread -------------------------------
    const int q = warp & 3;
    const int tn = p.bn;
    int lt = 0;
    for (int i = worker; i < num_items; i += workers, ++lt) {
      const Item t = item(i);
      const int b = lt & 1, u = lt >> 1;
      const bool ok = mbar_wait(&tfull[b], u & 1);
      if (!__all_sync(0xffffffffu, ok && !*abort_flag)) { *abort_flag = 1; break; }
      tc_fence_after();
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(b * kVlN);
      const int in_tile = rank * kVlM + 32 * q + lane, row = t.m0 + in_tile;
      const bool live = row < rows;
      const int ncol = min(tn, p.cols - t.n0);
      if constexpr (!GRAD) {
        const float ly = live ? p.ly[row] : 0.0f;
        const int yt = live ? p.target[row] - t.n0 : -1;
        const int y = (yt >= 0 && yt < ncol) ? yt : -1;          // the target's column, if it is here
        // the largest d (the target's own column is left out); a NaN shows in the sum below
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
            uint4* dst = reinterpret_cast<uint4*>(p.weights + row * p.pitch + t.n0 + c);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
          }
          __syncwarp();                          // the next tcgen05.ld is warp-wide
        }
        if (live) p.stats[static_cast<int64_t>(t.n0 / tn) * p.rows_max + row] = make_float2(shift, sum);
      } else {
        const bool whole = i < deal.full || deal.cuts == 1;
        const float f = whole && live ? p.factor[row] : 0.0f;
        __nv_bfloat16* out = p.out + static_cast<int64_t>(whole && live ? p.token[row] : 0) * p.cols + t.n0;
        float* part = whole ? nullptr : p.part + (static_cast<int64_t>(i - deal.full) * kVlM * C::CTAS + in_tile) * kVlN;
#pragma unroll 1
        for (int c = 0; c < ncol; c += 16) {
          uint32_t v[16];
          tmem_ld16(taddr + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < 2; ++h) {          // K % 8 == 0: whole groups of 8
            if (!live || c + 8 * h >= ncol) break;
            if (whole) {
              uint32_t o[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float x0 = __uint_as_float(v[8 * h + 2 * j]), x1 = __uint_as_float(v[8 * h + 2 * j + 1]);
                o[j] = f != 0.0f ? pack_bf16x2(x0 * f, x1 * f) : 0u;
              }
              *reinterpret_cast<uint4*>(out + c + 8 * h) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(part + c + 8 * h);
              dst[0] = make_uint4(v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3]);
              dst[1] = make_uint4(v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]);
            }
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(vl_peer(smem_u32(&tempty[b]), 0))
                       : "memory");
        else
          mbar_arrive(&tempty[b]);
      }
    }
  }

  // ------------------------------- teardown -------------------------------
  // every MMA of the pair, and the arrivals that its commits make in either CTA, are done
  if (warp == 1 && lane == 0 && !mbar_wait(drain, 0)) *abort_flag = 1;
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if (warp == 0 && lane == 0 && rank == 0)
      for (int it = (issued > ST ? issued - ST : 0); it < issued; ++it) mbar_wait_short(&full[it % ST], (it / ST) & 1);
    __syncthreads();
  }
  if constexpr (PAIR) vl_cluster_sync();    // neither CTA leaves while the other's copies, MMAs or arrivals reach it
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem_base) : "memory");
    else
      tmem_dealloc(tmem_base, 512);
  }
}
template <bool GRAD>
__global__ void __launch_bounds__(kVlThreads, 1)
    vl_gemm1_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA2,
                    const __grid_constant__ CUtensorMap tmB, const __grid_constant__ VlParams p) {
  vl_gemm<GRAD, false>(tmA, tmA2, tmB, p);
}
template <bool GRAD>
__global__ void __launch_bounds__(kVlThreads, 1) __cluster_dims__(2, 1, 1)
    vl_gemm2_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA2,
                    const __grid_constant__ CUtensorMap tmB, const __grid_constant__ VlParams p) {
  vl_gemm<GRAD, true>(tmA, tmA2, tmB, p);
}

// Numbers the tokens in the loss: one CTA, tokens in order. A token left out (ignored, or with a target outside
// the vocabulary, which the status word reports) has a loss of 0.
template <typename TI>
__global__ void __launch_bounds__(1024) vl_index_kernel(const TI* __restrict__ targets, int T, int64_t V, int64_t ignore,
                                                        int* __restrict__ token, int* __restrict__ target,
                                                        float* __restrict__ loss, int* __restrict__ count) {
  __shared__ int sm[32];
  __shared__ int base;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) base = 0;
  for (int t0 = 0; t0 < T; t0 += blockDim.x) {
    const int t = t0 + threadIdx.x;
    const int64_t y = t < T ? static_cast<int64_t>(targets[t]) : ignore;
    const bool in = t < T && y != ignore && y >= 0 && y < V;
    if (t < T && !in) {
      if (y != ignore) raise_status(kStatusTarget);
      loss[t] = 0.0f;
    }
    const unsigned votes = __ballot_sync(0xffffffffu, in);
    if (lane == 0) sm[warp] = __popc(votes);
    __syncthreads();
    int before = base + __popc(votes & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) before += sm[w];
    if (in) {
      token[before] = t;
      target[before] = static_cast<int>(y);
    }
    __syncthreads();
    if (threadIdx.x == blockDim.x - 1) base = before + (in ? 1 : 0);
    __syncthreads();
  }
  if (threadIdx.x == 0) *count = base;
}

// One warp per row of the piece: the target's logit in fp32, and the row's place in the packed copy where tokens
// are left out (packed: T, or 0 for no copy). Behind them, with dX, one warp per token of the whole call that
// zeroes the gradient of a token left out (found by its number: tokens in the loss are in order).
__global__ void __launch_bounds__(256) vl_target_kernel(const __nv_bfloat16* __restrict__ X,
                                                        const __nv_bfloat16* __restrict__ W, int K, int r0, int rows_max,
                                                        int T, const int* __restrict__ count,
                                                        const int* __restrict__ token, const int* __restrict__ target,
                                                        float* __restrict__ ly, __nv_bfloat16* __restrict__ packed,
                                                        __nv_bfloat16* __restrict__ dX) {
  const int lane = threadIdx.x & 31;
  const int i = static_cast<int>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  const int n = *count;
  if (i >= rows_max) {
    const int t = i - rows_max;
    if (!dX || t >= T || n == T) return;
    int lo = 0, hi = n;                  // the first number whose token is not before t
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (token[mid] < t) lo = mid + 1;
      else hi = mid;
    }
    if (lo < n && token[lo] == t) return;
    uint4* d = reinterpret_cast<uint4*>(dX + static_cast<int64_t>(t) * K);
    for (int c = lane; c < K / 8; c += 32) d[c] = make_uint4(0, 0, 0, 0);
    return;
  }
  if (i >= vl_rows(count, r0, rows_max)) return;
  const uint4* x = reinterpret_cast<const uint4*>(X + static_cast<int64_t>(token[r0 + i]) * K);
  const uint4* w = reinterpret_cast<const uint4*>(W + static_cast<int64_t>(target[r0 + i]) * K);
  uint4* to = n < T ? reinterpret_cast<uint4*>(packed + static_cast<int64_t>(i) * K) : nullptr;
  float acc = 0.0f;
#pragma unroll 4
  for (int c = lane; c < K / 8; c += 32) {
    const uint4 a = x[c], b = w[c];
    if (to) to[c] = a;
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
  if (lane == 0) ly[i] = acc;
}

// One warp per row of the piece. bn: words per tile of the logits.
__global__ void __launch_bounds__(256) vl_finish_kernel(const float2* __restrict__ stats, int r0, int rows_max, int tiles,
                                                        int bn, const int* __restrict__ count, const int* __restrict__ token,
                                                        const int* __restrict__ target, int V,
                                                        const float* __restrict__ dloss, int mean, float* __restrict__ loss,
                                                        __nv_bfloat16* weights, int64_t pitch, float* __restrict__ factor) {
  const int lane = threadIdx.x & 31;
  const int row = static_cast<int>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  if (row >= vl_rows(count, r0, rows_max)) return;
  float shift = 0.0f;                 // the row's: the largest of its tiles'
  for (int i = lane; i < tiles; i += 32) shift = fmaxf(shift, stats[static_cast<int64_t>(i) * rows_max + row].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) shift = fmaxf(shift, __shfl_xor_sync(0xffffffffu, shift, o));
  float z = 0.0f;
  for (int i = lane; i < tiles; i += 32) {
    const float2 s = stats[static_cast<int64_t>(i) * rows_max + row];
    z += shift > 0.0f ? s.y * expf(s.x - shift) : s.y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  const float one = shift > 0.0f ? expf(-shift) : 1.0f;
  const int t = token[r0 + row];
  if (lane == 0) loss[t] = shift > 0.0f ? shift + logf(z + one) : log1pf(z);
  if (!weights) return;
  __nv_bfloat16* w = weights + static_cast<int64_t>(row) * pitch;
  if (shift > 0.0f) {
    for (int v = lane; v < V; v += 32) {
      const float s = stats[static_cast<int64_t>(v / bn) * rows_max + row].x;
      if (s != shift) w[v] = __float2bfloat16_rn(__bfloat162float(w[v]) * expf(s - shift));
    }
    __syncwarp();
  }
  if (lane == 0) {
    w[target[r0 + row]] = __float2bfloat16_rn(-z);
    float g = dloss ? dloss[t] : 1.0f;
    if (mean) g /= static_cast<float>(*count);
    factor[row] = g / (z + one);
  }
}

// The tiles of dX that were cut: their partial sums in order. One CTA per tile and 16 of its rows.
template <int CTAS>
__global__ void __launch_bounds__(256) vl_reduce_kernel(const __grid_constant__ VlParams p, int workers) {
  constexpr int MT = kVlM * CTAS;
  const int rows = vl_rows(p.count, p.r0, p.rows_max);
  const int tiles_m = (rows + MT - 1) / MT;
  const VlDeal deal = vl_deal(tiles_m * p.tiles_n, workers, p.nkb);
  const int r = blockIdx.x, tile = deal.full + r;
  if (deal.cuts == 1 || r >= deal.rest) return;
  const int m0 = tile % tiles_m * MT, n0 = tile / tiles_m * p.bn;
  const int ncol = min(p.bn, p.cols - n0);
  for (int e = threadIdx.x; e < 16 * (kVlN / 8); e += blockDim.x) {
    const int in_tile = blockIdx.y * 16 + e / (kVlN / 8), row = m0 + in_tile, c = e % (kVlN / 8) * 8;
    if (row >= rows || c >= ncol) continue;
    float acc[8] = {};
#pragma unroll 4
    for (int w = 0; w < deal.cuts; ++w) {
      const float4* src = reinterpret_cast<const float4*>(
          p.part + (static_cast<int64_t>(w * deal.rest + r) * MT + in_tile) * kVlN + c);
      const float4 a = src[0], b = src[1];
      acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
      acc[4] += b.x; acc[5] += b.y; acc[6] += b.z; acc[7] += b.w;
    }
    const float f = p.factor[row];
    uint4 o = make_uint4(0, 0, 0, 0);
    if (f != 0.0f)
      o = make_uint4(pack_bf16x2(acc[0] * f, acc[1] * f), pack_bf16x2(acc[2] * f, acc[3] * f),
                     pack_bf16x2(acc[4] * f, acc[5] * f), pack_bf16x2(acc[6] * f, acc[7] * f));
    *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(p.token[row]) * p.cols + n0 + c) = o;
  }
}

// total = sum of the tokens' losses (fp64, fixed order), over their count for a mean (0 / 0 = NaN when no
// token is in the loss).
__global__ void __launch_bounds__(1024) vl_total_kernel(const float* __restrict__ loss, int64_t T, int mean,
                                                        const int* __restrict__ count, float* __restrict__ total) {
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
