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
//               K = 8192 a logit of 12 came out 1e-4 low), one CTA per row; copies the rows together where
//               tokens are left out, and zeroes those tokens' gradients;
//   vl_gemm<0>  logits tile by tile on the tensor cores (a CTA pair: 256 rows x up to 256 words, K in steps of 64
//               through a TMA-filled ring, two accumulators in tensor memory so the epilogue overlaps the next run);
//               epilogue: the fp32 sum of the tile's runs over K; exp(d_v) rounded to bf16 (the MMA operand of the gradient; a relative 2^-8 of each weight
//               at most) and its fp32 sum over the tile's words. Where a tile's largest d exceeds 40 its weights
//               are stored relative to that d (a shift per row and tile), so nothing overflows;
//   vl_finish   adds the tiles' sums in order, loss, the row's factor g / (1 + Z) and the target's g Z / (1 + Z);
//               brings a row whose tiles have shifts to one shift;
//   vl_gemm<1>  dX = weights x W (contraction over the vocabulary, W as the MN-major operand), times the row's
//               factor, less the target's share of W_y, both in fp32, rounded once to bf16. (With -Z among the bf16
//               weights its rounding alone was half of the gradient's error: 2.4e-3 against 1.7e-3 now, which is
//               the result's own rounding.) Whole waves of tiles run in step along the vocabulary, so W
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
constexpr int kVlStore = 32 * 32 * 2;      // 32 rows x 32 weights on their way out
template <bool PAIR> struct VlCfg {
  static constexpr int CTAS = PAIR ? 2 : 1;
  static constexpr int BROWS = kVlN / CTAS;           // words (or features) of a tile in one CTA's shared memory
  static constexpr int B_BYTES = BROWS * kVlK * 2;
  static constexpr int STAGE_BYTES = kVlABytes + B_BYTES;
  static constexpr int STAGES = PAIR ? 6 : 4;
  static constexpr int STORE_BYTES = 8 * kVlStore;          // a buffer per epilogue warp
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + STORE_BYTES + 256 + 1024;
  static_assert(SMEM_BYTES <= 227 * 1024 && (2 * STAGES + 5) * 8 + 8 <= 256, "shared memory per CTA");
};
constexpr int kVlThreads = 10 * 32;       // TMA, MMA, 8 epilogue warps
// The tensor cores drop what does not fit an accumulator's 24 bits, towards zero: in one run over K a logit loses a share of
// itself that grows with K and depends on the data (K = 8192, relative: features of random signs 8e-6, of one sign
// 3.4e-5, one large feature first 1.5e-5, last 0; of one sign at K = 2^20 6.7e-3). So a logit is the fp32 sum of near-equal
// runs of at most 16 blocks. Such a run of 64 steps loses between nothing (large features last, or zeros) and 2.1e-6 of
// itself (one sign), with random signs 1.06e-6: that middle is put back, 1.65e-8 a step, which leaves any data within
// 1.1e-6 at any K, and random signs within 2e-7. (Without it tokens of small losses, whose error is the logits' own, were
// up to 2.6e-6 off, one or two tokens of K = 6360.) Up to 8 blocks are one run as it is: 5e-7 at most where signs are
// random, and the epilogue binds there (with a factor on every logit 700 x 32000 x 64 took 39 us, not 35). The runs cost
// 1 to 4 % of a call; of 8 blocks 4 to 8 %.
constexpr int kVlRun = 16;
constexpr float kVlShort = 1.65e-8f;
constexpr float kVlMaxShift = 40.0f;      // exp(40) x any vocabulary stays far inside fp32 and bf16
constexpr unsigned kStatusTarget = 4u;

struct VlParams {
  const int* count;             // tokens in the loss
  int r0, rows_max;             // this piece: rows r0 .. of them, rows_max at most
  int copied;                   // <0>: rows live in the packed copy (second map) when count < copied
  int cols, bn;                 // columns (words, or features of dX) and columns per tile
  int tiles_n, nkb;             // column tiles; contraction blocks of 64
  int runs;                     // <0>: runs of blocks that are summed in fp32 (<1>: one)
  float run_scale;              // <0>: factor on every run, where there are several
  const __nv_bfloat16* w;       // <0>: W, for prefetches, and its row pitch
  int w_pitch;
  const int* target;            // <0>: per row
  const float* ly;              // <0>: target logits
  float2* stats;                // <0>: [half of a column tile][rows_max] (shift, sum)
  __nv_bfloat16* weights;       // <0>: [rows][pitch], or null (loss only)
  int64_t pitch;
  const int* token;             // <1>: the token of each row
  const float2* factor;         // <1>: per row, of the product and of W_y
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
__device__ __forceinline__ VlDeal vl_deal(int tiles, int workers, int nkb) {      // by a whole warp: a lane per cut
  VlDeal d;
  d.full = tiles / workers * workers;
  d.rest = tiles - d.full;
  int cuts = static_cast<int>(threadIdx.x & 31) + 1;
  float cost = 1e30f;
  if (cuts == 1 || (d.rest * cuts <= kVlParts * workers && cuts * 4 <= nkb + 3))
    cost = static_cast<float>((d.rest * cuts + workers - 1) / workers) * nkb / cuts +
           (cuts > 1 ? 0.25f * d.rest * cuts : 0.0f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float c = __shfl_xor_sync(0xffffffffu, cost, o);
    const int s = __shfl_xor_sync(0xffffffffu, cuts, o);
    if (c < cost || (c == cost && s < cuts)) { cost = c; cuts = s; }
  }
  d.cuts = cuts;
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

// 16 columns of this warp's lanes of tensor memory, written.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]),
      "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}

// Eight features of dX: factor.x x product - factor.y x W_y (a bf16 is the upper half of its fp32); a factor of 0
// takes nothing over from the row.
__device__ __forceinline__ uint4 vl_dx8(const float* acc, float2 f, uint4 w) {
  const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float lo = fmaf(-f.y, __uint_as_float(wv[j] << 16), acc[2 * j] * f.x);
    const float hi = fmaf(-f.y, __uint_as_float(wv[j] & 0xffff0000u), acc[2 * j + 1] * f.x);
    o[j] = f.x != 0.0f ? pack_bf16x2(lo, hi) : 0u;
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Every kernel of a call but the first is launched to start while the one before it runs: it lets the next one be
// set up in turn, and waits here before it touches anything that an earlier kernel of the call writes or reads. (A
// kernel is set up only once every CTA of the one before it has started, so a waiting CTA holds nobody up.)
__device__ __forceinline__ void vl_chain() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
  uint8_t* sE = base + ST * C::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sE + C::STORE_BYTES);
  uint64_t* empty = full + ST;
  uint64_t* tfull = empty + ST;            // [2]
  uint64_t* tempty = tfull + 2;            // [2]
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = PAIR ? blockIdx.x & 1 : 0;
  const int worker = PAIR ? blockIdx.x >> 1 : blockIdx.x, workers = PAIR ? gridDim.x >> 1 : gridDim.x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], 8 * C::CTAS); }
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
  if constexpr (!GRAD && !PAIR) {
    // Up to 128 rows are bound by reading W, an input of the call that no kernel of it writes: while the kernels
    // before this one run, the first 1.5 KB of every row of this CTA's tile come into L2.
    const int bytes = min(p.nkb * 128, 1536) & ~15;
    if (warp == 0 && p.w)
      for (int r = worker * p.bn + lane; r < min(p.cols, (worker + 1) * p.bn); r += 32)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p.w + static_cast<int64_t>(r) * p.w_pitch), "r"(min(bytes, p.w_pitch * 2))
                     : "memory");
    __syncwarp();
  }
  vl_chain();
  asm volatile("fence.proxy.async;" ::: "memory");     // what earlier kernels stored, for this one's TMA
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t idesc = idesc_bf16(kVlM * C::CTAS, 16, false, GRAD) - (2u << 17) + (static_cast<uint32_t>(p.bn >> 3) << 17);

  const int rows = vl_rows(p.count, p.r0, p.rows_max);
  const int tiles_m = (rows + kVlM * C::CTAS - 1) / (kVlM * C::CTAS);
  const int tiles = tiles_m * p.tiles_n;
  const VlDeal deal = GRAD ? vl_deal(tiles, workers, p.nkb) : VlDeal{tiles, 0, 1};
  const int num_items = deal.full + deal.rest * deal.cuts;
  const int bn_cta = p.bn / C::CTAS;
  // accumulator fills per item: the runs of a logit, near-equal ones; run r begins at block run_at(r)
  const int runs = GRAD ? 1 : p.runs;
  auto run_at = [&](int r) { return static_cast<int>(static_cast<int64_t>(p.nkb) * r / runs); };
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

  // A logits thread holds 128 sums: registers move from the first warpgroup to the epilogue's two. The launch has 168 a
  // thread, 3 x 168 = 504 per lane of the three; the split takes 64 + 2 x 216 = 496 of them.
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
              vl_tma<PAIR>(sB + s * C::B_BYTES + a * 8192, &tmB, bar, t.n0 + rank * bn_cta + 64 * a, kb * kVlK);
          }
        }
      }
      // This CTA's copies have landed once they are used. After a wait that gave up nobody uses them: then a limit far
      // above a copy's time stands for that. (A pair's copies count on the first CTA's barriers, but the second may have
      // run ahead of it, so neither CTA's copies can be told by those.)
      for (int last = max(it - ST, 0); last < it && mbar_wait_short(&empty[last % ST], (last / ST) & 1); ++last) {}
    }
  } else if (warp == 1) {
    // ------------------------------- MMA issuer (the first CTA) -------------------------------
    if (lane == 0 && rank == 0) {
      int it = 0, lt = 0;
      bool ok = true;
      for (int i = worker; i < num_items && ok; i += workers) {
        const Item t = item(i);
        for (int r = 0; r < runs && ok; ++r, ++lt) {
          const int b = lt & 1, u = lt >> 1;
          if (lt >= 2 && !mbar_wait(&tempty[b], (u - 1) & 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(b * kVlN);
          const int first = GRAD ? t.kb0 : run_at(r), last = GRAD ? t.kb1 : run_at(r + 1);
          for (int kb = first; kb < last; ++kb, ++it) {
            const int s = it % ST;
            if (!mbar_wait(&full[s], (it / ST) & 1) || *abort_flag) { ok = false; break; }
            tc_fence_after();
            const uint32_t a_addr = smem_u32(sA + s * kVlABytes), b_addr = smem_u32(sB + s * C::B_BYTES);
#pragma unroll
            for (int k = 0; k < kVlK / 16; ++k) {
              const uint64_t ad = sdesc_sw128(a_addr + 32u * k, 16u, 1024u);
              const uint64_t bd = GRAD ? sdesc_sw128(b_addr + 2048u * k, 8192u, 1024u)
                                       : sdesc_sw128(b_addr + 32u * k, 16u, 1024u);
              vl_mma<PAIR>(d, ad, bd, idesc, (kb > first || k > 0) ? 1u : 0u);
            }
            vl_commit<PAIR>(&empty[s]);
          }
          if (ok) vl_commit<PAIR>(&tfull[b]);
        }
      }
      if (!ok) *abort_flag = 1;
      vl_commit<PAIR>(drain);
    }
  } else {
    // ------------------ epilogue: one row and one half of the tile's columns per thread ------------------
    const int q = warp & 3, side = (warp - 2) >> 2, hn = p.bn / 2;
    const uint32_t out_buf = smem_u32(sE + (warp - 2) * kVlStore);
    const int tn = p.bn;
    int lt = 0;
    for (int i = worker; i < num_items; i += workers) {
      const Item t = item(i);
      const int in_tile = rank * kVlM + 32 * q + lane, row = t.m0 + in_tile;
      const bool live = row < rows;
      const int ncol = min(tn, p.cols - t.n0);
      float ly = 0.0f;
      int yt = -1;
      if (!GRAD && live) {             // on their way while the tile is computed
        ly = p.ly[row];
        yt = p.target[row] - t.n0;
      }
      const bool whole = GRAD && (i < deal.full || deal.cuts == 1);
      float2 f = make_float2(0.0f, 0.0f);
      uint4 wy[GRAD ? 16 : 1];         // the target's row of W, this thread's half of the tile
      if constexpr (GRAD) {
        if (whole && live) {
          f = p.factor[row];
          const uint4* src = reinterpret_cast<const uint4*>(p.w + static_cast<int64_t>(p.target[row]) * p.w_pitch + t.n0 + side * hn);
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (8 * k < min(ncol - side * hn, hn)) wy[k] = __ldg(src + k);
        }
      }
      uint32_t taddr = 0;
      auto filled = [&]() {            // wait for the next accumulator
        const int b = lt & 1, u = lt >> 1;
        const bool ok = mbar_wait(&tfull[b], u & 1);
        if (!__all_sync(0xffffffffu, ok && !*abort_flag)) { *abort_flag = 1; return false; }
        tc_fence_after();
        taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(b * kVlN);
        return true;
      };
      auto release = [&]() {           // the accumulator has been read
        const int b = lt & 1;
        ++lt;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(vl_peer(smem_u32(&tempty[b]), 0))
                         : "memory");
          else
            mbar_arrive(&tempty[b]);
        }
      };
      if constexpr (!GRAD) {
        // The sum of the runs, in order, takes the last one's place in tensor memory. (Kept in registers for the pass
        // below, 128 of them, it made that pass unrolled code that spills: 8192 x 32000 x 256 took 710 us, not 505.)
        if (runs == 1) {
          if (!filled()) break;
        } else {
          float acc[8][16] = {};
          bool ok = true;
#pragma unroll 1
          for (int r = 0; r < runs && ok; ++r) {
            ok = filled();
            if (!ok) break;
#pragma unroll
            for (int k = 0; k < 8; ++k) {          // columns past the tile's width hold nothing that is used
              uint32_t v[16];
              tmem_ld16(taddr + side * hn + 16 * k, v);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) acc[k][j] = fmaf(__uint_as_float(v[j]), p.run_scale, acc[k][j]);
            }
            if (r < runs - 1) release();
          }
          if (!ok) break;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (16 * k < hn) tmem_st16(taddr + side * hn + 16 * k, acc[k]);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        const int y = (yt >= 0 && yt < ncol) ? yt : -1;          // the target's column, if it is here
        // One pass against the target's logit, the target's own column left out; a second one, relative to the
        // half tile's largest d, only for the rare warp with a row whose weights could overflow. A NaN shows in the
        // sum. Chunks of 32 columns that are whole and hold no target of the warp's rows need no checks.
        const int c_end = min(ncol, (side + 1) * hn);
        float top = -INFINITY, shift = 0.0f, sum = 0.0f;
        while (true) {
          const float ref = ly + shift;
          float part[4] = {}, high[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int c = side * hn; c < c_end; c += 32) {
            uint32_t v[2][16];
            tmem_ld16(taddr + c, v[0]);
            tmem_ld16(taddr + c + 16, v[1]);
            const bool check = c + 32 > c_end || __any_sync(0xffffffffu, y >= c && y < c + 32);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (c + 16 * h >= c_end) break;
              float e[16];
              if (check) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const float l = __uint_as_float(v[h][j]);
                  const bool other = c + 16 * h + j < c_end && c + 16 * h + j != y;
                  if (other) high[j & 3] = fmaxf(high[j & 3], l);
                  e[j] = other ? __expf(l - ref) : 0.0f;
                }
              } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const float l = __uint_as_float(v[h][j]);
                  high[j & 3] = fmaxf(high[j & 3], l);
                  e[j] = __expf(l - ref);
                }
              }
#pragma unroll
              for (int j = 0; j < 16; ++j) part[j & 3] += e[j];
              if (p.weights) {
                uint32_t o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = pack_bf16x2(e[2 * j], e[2 * j + 1]);
                // 64-byte rows, 16-byte piece k of row r at k ^ (r / 2 % 4): no bank conflicts either way
                const uint32_t at = out_buf + 64u * lane, x = (lane >> 1) & 3;
                st_shared_v4(at + (((2 * h) ^ x) << 4), o[0], o[1], o[2], o[3]);
                st_shared_v4(at + (((2 * h + 1) ^ x) << 4), o[4], o[5], o[6], o[7]);
              }
            }
            if (p.weights) {                     // out in whole 64-byte runs of 8 rows at a time
              __syncwarp();
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int r = 8 * k + (lane >> 2), pc = lane & 3;
                uint4 o;
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
                             : "r"(out_buf + 64u * r + ((pc ^ ((r >> 1) & 3)) << 4)) : "memory");
                const int wr = row - lane + r;   // the pitch has room up to a multiple of 16 words
                if (wr < rows && c + 8 * pc < c_end)
                  *reinterpret_cast<uint4*>(p.weights + wr * p.pitch + t.n0 + c + 8 * pc) = o;
              }
            }
            __syncwarp();                        // the next tcgen05.ld is warp-wide
          }
          top = fmaxf(fmaxf(high[0], high[1]), fmaxf(high[2], high[3]));
          sum = (part[0] + part[1]) + (part[2] + part[3]);
          const bool far = shift == 0.0f && top - ly > kVlMaxShift;
          if (far) shift = top - ly;
          if (!__any_sync(0xffffffffu, far)) break;
        }
        release();                     // before the store below, which the arrival would wait for
        if (live) p.stats[static_cast<int64_t>(2 * (t.n0 / tn) + side) * p.rows_max + row] = make_float2(shift, sum);
      } else {
        if (!filled()) break;
        __nv_bfloat16* out = p.out + static_cast<int64_t>(whole && live ? p.token[row] : 0) * p.cols + t.n0;
        float* part = whole ? nullptr : p.part + (static_cast<int64_t>(i - deal.full) * kVlM * C::CTAS + in_tile) * kVlN;
        const int c_end = min(ncol, (side + 1) * hn);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int c = side * hn + 16 * k;
          if (c >= c_end) break;
          uint32_t v[16];
          tmem_ld16(taddr + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < 2; ++h) {          // K % 8 == 0: whole groups of 8
            if (!live || c + 8 * h >= c_end) break;
            if (whole) {
              *reinterpret_cast<uint4*>(out + c + 8 * h) = vl_dx8(reinterpret_cast<const float*>(v + 8 * h), f, wy[2 * k + h]);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(part + c + 8 * h);
              dst[0] = make_uint4(v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3]);
              dst[1] = make_uint4(v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]);
            }
          }
          __syncwarp();
        }
        release();
      }
    }
  }

  // ------------------------------- teardown -------------------------------
  // every MMA of the pair, and the arrivals that its commits make in either CTA, are done (again with a limit where
  // that wait gave up)
  if (warp == 1 && lane == 0 && !mbar_wait(drain, 0)) *abort_flag = 1;
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if (warp == 1 && lane == 0) mbar_wait_short(drain, 0);
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
                    const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ VlParams p) {
  vl_gemm<GRAD, false>(tmA, tmA2, tmB, p);
}
template <bool GRAD>
__global__ void __launch_bounds__(kVlThreads, 1) __cluster_dims__(2, 1, 1)
    vl_gemm2_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA2,
                    const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ VlParams p) {
  vl_gemm<GRAD, true>(tmA, tmA2, tmB, p);
}

// Numbers the tokens in the loss, in order: one CTA, 8192 tokens at a time. token[i] is the i-th of them, target[i]
// its target; the tokens left out (ignored, or with a target outside the vocabulary, which the status word
// reports) fill `token` from its end and have a loss of 0.
template <typename TI>
__global__ void __launch_bounds__(1024) vl_index_kernel(const TI* __restrict__ targets, int T, int64_t V, int64_t ignore,
                                                        int* __restrict__ token, int* __restrict__ target,
                                                        float* __restrict__ loss, int* __restrict__ count) {
  constexpr int PER = 8;
  __shared__ int sm[PER][32], all[PER];      // per 1024 tokens: each warp's count, then what lies before it; the sum
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int base = 0;
  for (int64_t t0 = 0; t0 < T; t0 += PER * 1024) {
    int64_t y[PER];
    unsigned votes[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int64_t t = t0 + 1024 * k + threadIdx.x;
      y[k] = t < T ? static_cast<int64_t>(targets[t]) : ignore;
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      votes[k] = __ballot_sync(0xffffffffu, y[k] != ignore && y[k] >= 0 && y[k] < V);
      if (lane == 0) sm[k][warp] = __popc(votes[k]);
    }
    __syncthreads();
    if (warp < PER) {
      const int mine = sm[warp][lane];
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      sm[warp][lane] = upto - mine;
      if (lane == 31) all[warp] = upto;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int64_t t = t0 + 1024 * k + threadIdx.x;
      const int before = base + sm[k][warp] + __popc(votes[k] & ((1u << lane) - 1u));
      if (votes[k] >> lane & 1u) {
        token[before] = static_cast<int>(t);
        target[before] = static_cast<int>(y[k]);
      } else if (t < T) {
        if (y[k] != ignore) raise_status(kStatusTarget);
        token[T - 1 - (t - before)] = static_cast<int>(t);
        loss[t] = 0.0f;
      }
      base += all[k];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) *count = base;
}

// Four warps per row of the piece: the target's logit in fp32, and the row's place in the packed copy where tokens
// are left out. Behind them, with dX, four warps per token left out of the whole call, which zero its gradient.
constexpr int kVlRowThreads = 128;
__global__ void __launch_bounds__(kVlRowThreads) vl_target_kernel(const __nv_bfloat16* __restrict__ X,
                                                                  const __nv_bfloat16* __restrict__ W, int K, int r0,
                                                                  int rows_max, int T, const int* __restrict__ count,
                                                                  const int* __restrict__ token,
                                                                  const int* __restrict__ target, float* __restrict__ ly,
                                                                  __nv_bfloat16* __restrict__ packed,
                                                                  __nv_bfloat16* __restrict__ dX) {
  __shared__ float sm[kVlRowThreads / 32];
  vl_chain();
  const int lane = threadIdx.x & 31, i = blockIdx.x;
  const int n = *count;
  if (i >= rows_max) {
    if (!dX || n + (i - rows_max) >= T) return;
    const int t = token[n + (i - rows_max)];
    uint4* d = reinterpret_cast<uint4*>(dX + static_cast<int64_t>(t) * K);
    for (int c = threadIdx.x; c < K / 8; c += kVlRowThreads) d[c] = make_uint4(0, 0, 0, 0);
    return;
  }
  if (i >= vl_rows(count, r0, rows_max)) return;
  const uint4* x = reinterpret_cast<const uint4*>(X + static_cast<int64_t>(token[r0 + i]) * K);
  const uint4* w = reinterpret_cast<const uint4*>(W + static_cast<int64_t>(target[r0 + i]) * K);
  uint4* to = n < T ? reinterpret_cast<uint4*>(packed + static_cast<int64_t>(i) * K) : nullptr;
  float acc = 0.0f;
#pragma unroll 8
  for (int c = threadIdx.x; c < K / 8; c += kVlRowThreads) {
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
  if (lane == 0) sm[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) ly[i] = (sm[0] + sm[1]) + (sm[2] + sm[3]);
}

// 32 rows per CTA: lanes are rows (the statistics of 32 rows of a tile are one run of memory), warps share the tiles;
// their sums are added in warp order. tiles, bn: half tiles of the logits and their words.
constexpr int kVlFinishThreads = 1024;
__global__ void __launch_bounds__(kVlFinishThreads) vl_finish_kernel(const float2* __restrict__ stats, int r0, int rows_max, int tiles,
                                                        int bn, const int* __restrict__ count, const int* __restrict__ token,
                                                        int V,
                                                        const float* __restrict__ dloss, int mean, float* __restrict__ loss,
                                                        __nv_bfloat16* weights, int64_t pitch, float2* __restrict__ factor) {
  constexpr int W = kVlFinishThreads / 32;
  __shared__ float2 sm[W][32];
  __shared__ float row_shift[32];
  vl_chain();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = static_cast<int>(blockIdx.x) * 32 + lane, n = *count, rows = max(0, min(rows_max, n - r0));
  const bool live = row < rows;
  const int t = live ? token[r0 + row] : 0;
  float g = live && dloss ? dloss[t] : 1.0f;
  // (shift, sum relative to exp(shift)) of this warp's tiles
  auto add = [](float2& a, float2 b) {
    if (b.x > a.x) {
      a.y = a.y * expf(a.x - b.x) + b.y;
      a.x = b.x;
    } else {
      a.y += b.x < a.x ? b.y * expf(b.x - a.x) : b.y;
    }
  };
  float2 a = make_float2(0.0f, 0.0f);
  if (live) {
    for (int i = warp; i < tiles; i += 8 * W) {
      float2 b[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        b[k] = i + k * W < tiles ? stats[static_cast<int64_t>(i + k * W) * rows_max + row] : make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < 8; ++k) add(a, b[k]);
    }
  }
  sm[warp][lane] = a;
  __syncthreads();
  if (warp < 4) {                     // 8 warps' sums each, then those 4
#pragma unroll
    for (int w = 1; w < W / 4; ++w) add(a, sm[warp + 4 * w][lane]);
    sm[warp][lane] = a;
  }
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < 4; ++w) add(a, sm[w][lane]);
    row_shift[lane] = a.x;
    if (live) {
      const float one = a.x > 0.0f ? expf(-a.x) : 1.0f;
      loss[t] = a.x > 0.0f ? a.x + logf(a.y + one) : log1pf(a.y);
      if (weights) {
        if (mean) g /= static_cast<float>(n);
        g /= a.y + one;
        factor[row] = make_float2(g, g * a.y);
      }
    }
  }
  if (!weights) return;
  __syncthreads();
  // rows with shifts: every weight relative to the row's (rare: a target 40 below another word)
  for (int i = 0; i < 32; ++i) {
    const float shift = row_shift[i];
    const int r = static_cast<int>(blockIdx.x) * 32 + i;
    if (!(shift > 0.0f) || r >= rows) continue;
    __nv_bfloat16* w = weights + static_cast<int64_t>(r) * pitch;
    for (int v = threadIdx.x; v < V; v += blockDim.x) {
      const float s = stats[static_cast<int64_t>(v / bn) * rows_max + r].x;
      if (s != shift) w[v] = __float2bfloat16_rn(__bfloat162float(w[v]) * expf(s - shift));
    }
  }
}

// The tiles of dX that were cut: their partial sums in order. One CTA per tile and 8 of its rows.
template <int CTAS>
__global__ void __launch_bounds__(256) vl_reduce_kernel(const __grid_constant__ VlParams p, int workers) {
  constexpr int MT = kVlM * CTAS;
  vl_chain();
  const int rows = vl_rows(p.count, p.r0, p.rows_max);
  const int tiles_m = (rows + MT - 1) / MT;
  const VlDeal deal = vl_deal(tiles_m * p.tiles_n, workers, p.nkb);
  const int r = blockIdx.x, tile = deal.full + r;
  if (deal.cuts == 1 || r >= deal.rest) return;
  const int m0 = tile % tiles_m * MT, n0 = tile / tiles_m * p.bn;
  const int ncol = min(p.bn, p.cols - n0);
  const int in_tile = blockIdx.y * 8 + threadIdx.x / (kVlN / 8), row = m0 + in_tile, c = threadIdx.x % (kVlN / 8) * 8;
  if (row >= rows || c >= ncol) return;
  float acc[8] = {};
#pragma unroll 8
  for (int w = 0; w < deal.cuts; ++w) {
    const float4* src = reinterpret_cast<const float4*>(
        p.part + (static_cast<int64_t>(w * deal.rest + r) * MT + in_tile) * kVlN + c);
    const float4 a = src[0], b = src[1];
    acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
    acc[4] += b.x; acc[5] += b.y; acc[6] += b.z; acc[7] += b.w;
  }
  const uint4 w = __ldg(reinterpret_cast<const uint4*>(p.w + static_cast<int64_t>(p.target[row]) * p.w_pitch + n0 + c));
  *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(p.token[row]) * p.cols + n0 + c) = vl_dx8(acc, p.factor[row], w);
}

// total = sum of the tokens' losses (fp64, fixed order), over their count for a mean (0 / 0 = NaN when no
// token is in the loss).
__global__ void __launch_bounds__(1024) vl_total_kernel(const float* __restrict__ loss, int64_t T, int mean,
                                                        const int* __restrict__ count, float* __restrict__ total) {
  __shared__ double sm[32];
  vl_chain();
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
