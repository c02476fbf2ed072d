// Y = X W^T for a few tokens (T <= 64) and a 4-bit weight with one fp32 constant per block of 64:
//     W[n][k] = level[code[n][k]] * absmax[n][k / 64],   any codebook of up to 16 levels.
//
// HBM bounds it at a few tokens: 0.5625 B per weight, read once. The contraction runs on mma.sync m16n8k16 (the
// weight as the 16-row A operand, X as the 8-token B operand; a 128-row tensor-memory tile would be padding at
// these token counts). One shared-memory load turns a code byte into the bf16 pair (level[high], level[low]):
// a 256-entry table, one copy per lane so the lookups have no bank conflicts. Inside a block of 64 the MMA's k
// index is permuted alike on both operands, so lane j of a quad holds elements 16 j .. 16 j + 15: 8 code bytes and
// 32 bytes of X in a row. The block's constant multiplies the fp32 result of its four MMAs, so the only rounding
// of a weight is its level's to bf16 (a relative 2^-8 at most). The host picks a common factor for the levels under
// which they round best (int4's sevenths become exact), and the fp32 sums are divided by it at the end. Distance from
// the 64-bit result (2-norm), of which the rounding of the result alone is 1.6e-3: NF4 at 8192 x 8192 1.9e-3 to
// 2.0e-3 (2.1e-3 with the levels as they are), int4 with 16 tokens 1.7e-3 (2.3e-3).
// Two kernels: one for one or two tokens, one for up to 16 (more run as groups of 16, whose weights after the first
// come from L2 where they fit). In both every warp streams its own share of a CTA's rows or contraction with no
// barrier between warps, and fp32 sums are added in a fixed order: deterministic.
#pragma once

#include "codec.cuh"
#include "common.cuh"
#include "decode_nf4.cuh"

namespace qnf4 {

constexpr int kClMaxTokens = 64;
// Measured (six weights in turn, replayed back to back): 22016 x 8192 at one token 23 us (4.4 TB/s), 4 tokens 27, 16
// tokens 39, 17 to 32 tokens 69 to 74, 64 tokens 145 (every group of 16 looks the weight up again); 8192 x 8192 12, 13,
// 17, 31, 59 us. The plain copy's rate would be 15.5 and 5.8 us.
//
// Shared memory: the table (256 entries of 256 bytes, the lane copies in the first 128) sits at shared address
// 64 KB, so one byte permute forms a lookup's address; the stream's slots lie above it, sums (and X) below.
constexpr uint32_t kClTable = 1u << 16;
constexpr int kClBaseMax = 4096;         // where the dynamic shared memory may begin, at most

struct ClParams {
  int T, N, nkb, tiles, workers;         // tiles of rows, and the CTAs (or pairs) that share them
  const __nv_bfloat16* X;
  const uint8_t* codes;
  const float* absmax;
  float unscale;                         // the table holds levels / unscale
  __nv_bfloat16* Y;
};

__device__ __forceinline__ void cl_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Store to the same shared address in CTA `rank` of the cluster.
__device__ __forceinline__ void cl_st_peer(uint32_t addr, uint32_t rank, float v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.f32 [a], %2;\n\t}" ::"r"(addr),
      "r"(rank), "f"(v)
      : "memory");
}
__device__ __forceinline__ float cl_lds(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cl_sts2(uint32_t addr, float a, float b) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

// ---- one or two tokens ---------------------------------------------------------------------------------
// Lookups, X and the codes all pass through the SM's one shared-memory pipe, and with one token that pipe binds
// as soon as HBM does; so the stream takes as little of it, and as few instructions, as it can. TMA brings units of
// 8 rows x 256 bytes of codes (two windows of 256 elements, 4 blocks) and their 64 constants into two slots that
// every warp keeps for itself (no barrier with another warp; 64 KB per SM in flight), refilled as soon as the
// warp has read them into registers. A warp reads a window with two conflict-free 16-byte loads: lane l has chunk
// l % 8 of row l / 8 and of that row + 4. In the MMA each quad of lanes is then half a row (chunks 0..3 or 4..7: 128
// elements), so the 16 rows of the A operand are 8 weight rows x 2 halves h, and the 8 columns of B keep the halves
// and the two blocks e inside each apart: column 4 t + 2 h + e is x of token t and half h, zero except where lane j holds block e = j / 2 (those lanes' registers stay zero:
// they take no part in the load). Lane (g, j) with g = 2 r + h finds the sums of blocks 2 h and 2 h + 1 of row r
// (and r + 4) and token t in its own accumulators where j = 2 t + h. A CTA owns a run of 8-row tiles, cut evenly
// over its warps. (Loads into registers 4 windows ahead took 39 us for 22016 x 8192: the lookups' waits shared
// scoreboards with the loads in flight.)
constexpr int kC1Warps = 16;              // 12 to 20 measure alike: the shared-memory pipe binds, not latency
constexpr int kC1Ring = 2;
constexpr int kC1Pass = 64;               // tiles per pass
constexpr int kC1Seg = kC1Pass / kC1Warps + 2;
constexpr int kC1Tokens = 2;
constexpr int kC1CodeBytes = 8 * 256, kC1ScaleBytes = 8 * 8 * 4, kC1SlotBytes = kC1CodeBytes + kC1ScaleBytes;
constexpr uint32_t kC1Slots = 2u << 16;   // above the table: the warps' slots, then their barriers
constexpr uint32_t kC1Bars = kC1Slots + kC1Warps * kC1Ring * kC1SlotBytes;
constexpr int kC1Smem = static_cast<int>(kC1Bars) + kC1Warps * kC1Ring * 8;
constexpr int kC1RedBytes = kC1Warps * kC1Seg * 32 * 4;       // below it: the warps' sums, then X
constexpr int kC1XBytes = 65536 - kClBaseMax - kC1RedBytes;
static_assert(kC1Smem <= 227 * 1024 && kC1SlotBytes % 128 == 0 && kC1RedBytes % 128 == 0, "shared memory");
static_assert(kC1Ring == 2, "the slot and its phase are tracked as one toggle each");
__host__ __device__ constexpr int64_t c1_x_bytes(int64_t T, int64_t nkb) { return T * ((nkb + 7) / 8 * 1024); }

__device__ __forceinline__ void c1_tma(uint32_t dst, const void* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void c1_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// One fp32 (or a zero) global -> shared, and this thread's arrival on `bar` once its copies so far are complete.
__device__ __forceinline__ void c1_cp4(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void c1_cp_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void c1_ldx(uint4& x, uint32_t addr, uint32_t on) {   // lanes without x keep their zeros
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t@p ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "+r"(x.x), "+r"(x.y), "+r"(x.z), "+r"(x.w)
      : "r"(addr), "r"(on));
}
__device__ __forceinline__ void c1_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// VEC: rows of constants are 16-byte aligned (K % 256 == 0) and come by TMA too; otherwise by 4-byte copies.
template <bool VEC>
__global__ void __launch_bounds__(kC1Warps * 32, 1)
    codebook_linear1_kernel(const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmS,
                            const __grid_constant__ ClParams p, const __grid_constant__ CodebookArg cb) {
  extern __shared__ __align__(1024) uint8_t cl_smem[];
  const uint32_t base = smem_u32(cl_smem), window = base & 0xFF000000u;
  const uint32_t table = window | kClTable, xs = base + kC1RedBytes;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, j = lane & 3;
  if (base - window > kClBaseMax) {
    if (threadIdx.x == 0) raise_status(kStatusTimeout);
    return;
  }
  const uint32_t slots = (window | kC1Slots) + warp * kC1Ring * kC1SlotBytes;
  const uint32_t bars = (window | kC1Bars) + warp * kC1Ring * 8;
  if (lane == 0) {
    for (int s = 0; s < kC1Ring; ++s)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bars + 8 * s), "r"(VEC ? 1 : 33));
    fence_barrier_init();
  }
  const int nu = (p.nkb + 7) / 8;                // units per row
  for (int i = threadIdx.x; i < 256 * 32; i += blockDim.x) {
    const uint32_t v = pack_bf16x2(cb.levels[i >> 9], cb.levels[(i >> 5) & 15]);
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(table + (static_cast<uint32_t>(i >> 5) << 8) + 4u * (i & 31)), "r"(v)
                 : "memory");
  }
  // All of the above reads nothing of the kernel before this one in the stream and may run beside its end; the
  // next kernel may do the same beside this one's.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncwarp();
  const uint32_t lanebyte = table | (4u * lane);

  // B operand: column g = 4 t + 2 h + e; this lane's 32 elements of half h, if they are of block e
  const int bt = g >> 2;
  const uint32_t on = (bt < p.T && (j >> 1) == (g & 1)) ? 1u : 0u;
  const uint32_t x_base = xs + 1024u * (bt * nu) + 16u * (4 * ((g >> 1) & 1) + j);
  // A operand: 16 bytes of row l / 8 (and that + 4); its blocks of a window begin at 2 h
  const int ar = lane >> 3, h = (lane >> 2) & 1;
  const uint32_t code_off = 256u * ar + 16u * (lane & 7), scale_off = kC1CodeBytes + 32u * ar + 8u * h;
  uint4 x[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) x[q] = make_uint4(0, 0, 0, 0);

  const int t_lo = static_cast<int>(static_cast<int64_t>(blockIdx.x) * p.tiles / gridDim.x);
  const int t_hi = static_cast<int>(static_cast<int64_t>(blockIdx.x + 1) * p.tiles / gridDim.x);
  uint32_t in_slot = 0, slot = 0, phase = 0;     // the slots to fill and to read next
  auto stage_x = [&]() {
    // X window by window, padded with zeros: 16-byte piece q of (half h, lane j) at 128 q + 16 (4 h + j)
    for (int i = threadIdx.x; i < p.T * nu * 64; i += blockDim.x) {
      const int t = i / (nu * 64), c = i - t * nu * 64;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (c < p.nkb * 8) v = __ldg(reinterpret_cast<const uint4*>(p.X + static_cast<int64_t>(t) * p.nkb * 64) + c);
      st_shared_v4(xs + 512u * (t * nu * 2 + (c >> 5)) + 128u * (c & 3) + 16u * ((c >> 2) & 7), v.x, v.y, v.z, v.w);
    }
    __syncthreads();
  };
  bool ok = true;
  for (int t0 = t_lo; t0 < t_hi; t0 += kC1Pass) {
    const int nt = min(kC1Pass, t_hi - t0);
    const int total = nt * nu, chunk = (total + kC1Warps - 1) / kC1Warps;
    const int b0 = min(total, warp * chunk), n = min(total, b0 + chunk) - b0;
    int issued = 0, i = 0;
    if (n == 0 && t0 == t_lo) stage_x();
    if (n > 0) {
      int ck = b0 % nu, seg = 0;                 // the unit to read next
      int lk = ck, row = (t0 + b0 / nu) * 8;     // the unit to fetch next
      auto fetch = [&]() {
        const uint32_t dst = slots + in_slot * kC1SlotBytes, bar = bars + 8 * in_slot;
        if constexpr (!VEC) {
#pragma unroll
          for (int e = lane; e < 64; e += 32) {
            const int r = row + (e >> 3), kb = lk * 8 + (e & 7);
            const bool in = r < p.N && kb < p.nkb;
            c1_cp4(dst + kC1CodeBytes + 4u * e, p.absmax + (in ? static_cast<int64_t>(r) * p.nkb + kb : 0), in ? 4u : 0u);
          }
          c1_cp_arrive(bar);
        }
        if (lane == 0) {
          c1_expect(bar, VEC ? kC1SlotBytes : kC1CodeBytes);
          c1_tma(dst, &tmC, bar, lk * 256, row);
          if constexpr (VEC) c1_tma(dst + kC1CodeBytes, &tmS, bar, lk * 8, row);
        }
        in_slot ^= 1;
        ++issued;
        if (++lk == nu) { lk = 0; row += 8; }
      };
      fetch();
      if (n > 1) fetch();
      if (t0 == t_lo) stage_x();      // while the first units are on their way
      uint32_t xa = x_base + 1024u * ck;
      float acc0 = 0.0f, acc1 = 0.0f;
      auto flush = [&]() {      // rows r and r + 4 of token t = j / 2, half h = j % 2 (where that is this lane's)
        if ((j & 1) == h) {
          const uint32_t red = base + static_cast<uint32_t>((warp * kC1Seg + seg) * 128) + 4u * (j >> 1);
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(red + 8u * (2 * ar + h)), "f"(acc0) : "memory");
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(red + 8u * (2 * (ar + 4) + h)), "f"(acc1) : "memory");
        }
        acc0 = acc1 = 0.0f;
        ++seg;
      };
      for (; i < n; ++i) {
        if (!__all_sync(0xffffffffu, ok && mbar_wait_addr(bars + 8 * slot, phase))) { ok = false; break; }
        const uint32_t at = slots + slot * kC1SlotBytes;
        uint4 w[4];
        float2 sc[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {            // window u / 2, rows + 4 (u % 2)
          w[u] = dc_ld128(at + code_off + 1024u * (u & 1) + 128u * (u >> 1));
          sc[u] = dc_ldf2(at + scale_off + 128u * (u & 1) + 16u * (u >> 1));
        }
        __syncwarp();           // the slot has been read
        slot ^= 1;
        phase ^= slot ^ 1;
        if (issued < n) fetch();
#pragma unroll
        for (int u = 0; u < 4; u += 2) {
#pragma unroll
          for (int q = 0; q < 4; ++q) c1_ldx(x[q], xa + 256u * u + 128u * q, on);
          float d0[4] = {}, d1[4] = {};
#pragma unroll
          for (int q = 0; q < 4; ++q) {          // 8 elements of the lane's 32 at a time: one word of codes
            const uint32_t u0 = dc_word(w[u], q), u1 = dc_word(w[u + 1], q);
            c1_mma(d0, dc_pair<0>(u0, lanebyte), dc_pair<0>(u1, lanebyte), dc_pair<1>(u0, lanebyte), dc_pair<1>(u1, lanebyte),
                   x[q].x, x[q].y);
            c1_mma(d1, dc_pair<2>(u0, lanebyte), dc_pair<2>(u1, lanebyte), dc_pair<3>(u0, lanebyte), dc_pair<3>(u1, lanebyte),
                   x[q].z, x[q].w);
          }
          acc0 = fmaf(sc[u].x, d0[0] + d1[0], fmaf(sc[u].y, d0[1] + d1[1], acc0));
          acc1 = fmaf(sc[u + 1].x, d0[2] + d1[2], fmaf(sc[u + 1].y, d0[3] + d1[3], acc1));
        }
        xa += 1024;
        if (++ck == nu) {
          ck = 0;
          xa = x_base;
          flush();
        }
      }
      if (ok && ck != 0) flush();
      for (; i < issued; ++i) {      // after a wait that gave up: wait shortly for this warp's copies in flight
        mbar_wait_short_addr(bars + 8 * slot, phase);
        slot ^= 1;
        phase ^= slot ^ 1;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < nt * 8 * p.T; e += blockDim.x) {
      const int tile = e / (8 * p.T), r = e / p.T % 8, t = e % p.T;
      const int first = tile * nu / chunk, last = ((tile + 1) * nu - 1) / chunk;
      float sum = 0.0f;
      for (int v = first; v <= last; ++v) {
        const uint32_t red = base + static_cast<uint32_t>((v * kC1Seg + tile - (v * chunk) / nu) * 128) + 16u * r + 4u * t;
        sum += cl_lds(red) + cl_lds(red + 8u);
      }
      const int out = (t0 + tile) * 8 + r;
      if (out < p.N) p.Y[static_cast<int64_t>(t) * p.N + out] = __float2bfloat16_rn(sum * p.unscale);
    }
    __syncthreads();
  }
}

// ---- up to 16 tokens ------------------------------------------------------------------------------------
// X no longer fits beside the stream, and reading its fragments once per 16 rows would cost the shared-memory
// pipe more than the lookups do. So a warp keeps the fragments of 256 elements of all tokens in registers (64 of
// them for 16 tokens) and runs up to 4 tiles of 16 rows past them, with their accumulators in registers too. A
// CTA owns a run of row tiles; its warps each have their own share of the contraction, and their sums meet at the
// end of a pass of 4 tiles, while the next pass's codes are on their way. (Few tiles: a CTA pair shares one tile's
// contraction.) Codes and constants of one or two tiles and 256 elements come by TMA into two slots per warp
// (32 rows x 128 bytes, 128-byte swizzle; quad g takes row 2 (g % 4) + g / 4 of each 8, whose 8-byte
// loads then hit distinct banks). (Boxes of 16 rows x 64 or 128 bytes with 4-byte copies of the constants took
// 51 us for 16 tokens through 8192 x 22016, 32 us of it for the stream alone.)
constexpr int kC4Tiles = 4;
constexpr uint32_t kC4Slots = 2u << 16;
template <int NT> struct C4 {
  static constexpr int WARPS = NT == 1 ? 16 : 8, ST = NT == 1 ? 1 : 2;      // warps; tiles per slot
  static constexpr int CODE_BYTES = ST * 16 * 128, SCALE_BYTES = ST * 16 * 4 * 4;
  static constexpr uint32_t SCALES = kC4Slots + WARPS * 2 * CODE_BYTES, BARS = SCALES + WARPS * 2 * SCALE_BYTES;
  static constexpr int SMEM = static_cast<int>(BARS) + WARPS * 2 * 8;
  static constexpr int SUM_BYTES = kC4Tiles * 16 * 8 * NT * 4;              // a warp's sums of a pass
  static_assert(SMEM <= 227 * 1024 && kClBaseMax + (WARPS + 1) * SUM_BYTES <= 65536, "shared memory");
};

// VEC: constants by TMA (K % 256 == 0), else by 4-byte copies.
template <int NT, bool VEC, bool PAIR>
__device__ __forceinline__ void codebook_linear4(const CUtensorMap& tmC, const CUtensorMap& tmS, const ClParams& p,
                                                 const CodebookArg& cb) {
  const int tok0 = blockIdx.y * 8 * NT, T = min(8 * NT, p.T - tok0);        // this group of tokens
  using C = C4<NT>;
  constexpr int TT = 8 * NT, WARPS = C::WARPS, ST = C::ST;
  extern __shared__ __align__(1024) uint8_t cl_smem[];
  const uint32_t base = smem_u32(cl_smem), window = base & 0xFF000000u;
  const uint32_t table = window | kClTable;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, j = lane & 3;
  const int rank = PAIR ? blockIdx.x & 1 : 0, worker = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  if (base - window > kClBaseMax) {
    if (threadIdx.x == 0) raise_status(kStatusTimeout);
    return;
  }
  const uint32_t slots = (window | kC4Slots) + warp * 2 * C::CODE_BYTES;
  const uint32_t scales = window + C::SCALES + warp * 2 * C::SCALE_BYTES;
  const uint32_t bars = window + C::BARS + warp * 2 * 8;
  const uint32_t red = base + C::SUM_BYTES;     // the warps' sums; the pair's second half hands over at base
  if (lane == 0) {
    for (int s = 0; s < 2; ++s)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bars + 8 * s), "r"(VEC ? 1 : 33));
    fence_barrier_init();
  }
  for (int i = threadIdx.x; i < 256 * 32; i += blockDim.x) {
    const uint32_t v = pack_bf16x2(cb.levels[i >> 9], cb.levels[(i >> 5) & 15]);
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(table + (static_cast<uint32_t>(i >> 5) << 8) + 4u * (i & 31)), "r"(v)
                 : "memory");
  }
  if constexpr (PAIR) cl_cluster_sync();
  else __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");     // as in the kernel above
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncwarp();
  const uint32_t lanebyte = table | (4u * lane);
  const int gr = 2 * (g & 3) + (g >> 2);             // quad g's row of each 8

  const int t_lo = static_cast<int>(static_cast<int64_t>(worker) * p.tiles / p.workers);
  const int t_hi = static_cast<int>(static_cast<int64_t>(worker + 1) * p.tiles / p.workers);
  constexpr int PARTS = (PAIR ? 2 : 1) * WARPS;
  const int part = rank * WARPS + warp;              // this warp's share of the contraction
  const int units = (p.nkb + 3) / 4;                 // of 256 elements
  const int u_lo = part * units / PARTS, nu = (part + 1) * units / PARTS - u_lo;
  uint32_t in_slot = 0, slot = 0, phase = 0;
  bool ok = true;
  // everything this warp streams, over all passes: pass (tiles ft0 .. + 3), unit, group of ST tiles
  const int total = nu * ((t_hi - t_lo) / kC4Tiles * (kC4Tiles / ST) + ((t_hi - t_lo) % kC4Tiles + ST - 1) / ST);
  // CTAs begin at different units of their warps' shares, so that they do not all ask L2 for the same lines of X at
  // once
  const int rot = nu > 0 ? static_cast<int>(blockIdx.x) % nu : 0;
  int issued = 0, done = 0, ft0 = t_lo, fu = rot, fn = 0, fh = 0;
  auto fetch = [&]() {
    const uint32_t bar = bars + 8 * in_slot, sdst = scales + in_slot * C::SCALE_BYTES;
    const int row = (ft0 + ST * fh) * 16;
    if constexpr (!VEC) {
#pragma unroll
      for (int e = lane; e < ST * 64; e += 32) {
        const int r = row + (e >> 2), kb = 4 * (u_lo + fu) + (e & 3);
        const bool in = r < p.N && kb < p.nkb;
        c1_cp4(sdst + 4u * e, p.absmax + (in ? static_cast<int64_t>(r) * p.nkb + kb : 0), in ? 4u : 0u);
      }
      c1_cp_arrive(bar);
    }
    if (lane == 0) {
      c1_expect(bar, C::CODE_BYTES + (VEC ? C::SCALE_BYTES : 0));
      c1_tma(slots + in_slot * C::CODE_BYTES, &tmC, bar, (u_lo + fu) * 128, row);
      if constexpr (VEC) c1_tma(sdst, &tmS, bar, (u_lo + fu) * 4, row);
    }
    in_slot ^= 1;
    ++issued;
    if (ST * ++fh >= min(kC4Tiles, t_hi - ft0)) {
      fh = 0;
      if (++fu == nu) fu = 0;
      if (++fn == nu) { fn = 0; ft0 += kC4Tiles; }
    }
  };
  if (total > 0) fetch();
  if (total > 1) fetch();
  uint4 x[4][NT][2];           // the fragments of a unit
  for (int t0 = t_lo; t0 < t_hi; t0 += kC4Tiles) {
    const int nt = min(kC4Tiles, t_hi - t0);
    float acc[kC4Tiles][NT][4] = {};
    for (int un = 0; un < nu && ok; ++un) {
      const int u = un + rot < nu ? un + rot : un + rot - nu;
      if (nu > 1 || t0 == t_lo) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            x[b][m][0] = x[b][m][1] = make_uint4(0, 0, 0, 0);
            const int kb = 4 * (u_lo + u) + b;
            if (8 * m + g < T && kb < p.nkb) {
              const uint4* xp = reinterpret_cast<const uint4*>(p.X + (static_cast<int64_t>(tok0 + 8 * m + g) * p.nkb + kb) * 64 + 16 * j);
              x[b][m][0] = __ldg(xp);
              x[b][m][1] = __ldg(xp + 1);
            }
          }
      }
#pragma unroll
      for (int t = 0; t < kC4Tiles; ++t) {
        if (t >= nt || !ok) break;
        if (t % ST == 0 && !__all_sync(0xffffffffu, mbar_wait_addr(bars + 8 * slot, phase))) { ok = false; break; }
        const uint32_t at = slots + slot * C::CODE_BYTES + 2048u * (t % ST) + 128u * gr + 8u * (j & 1);
        const uint32_t sa = scales + slot * C::SCALE_BYTES + 256u * (t % ST) + 16u * gr;
        uint2 w[4][2];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t c = at + (static_cast<uint32_t>((2 * b + (j >> 1)) ^ gr) << 4);
          w[b][0] = dc_ld64(c);
          w[b][1] = dc_ld64(c + 1024);
        }
        const uint4 f0 = dc_ld128(sa), f1 = dc_ld128(sa + 128);
        if (t % ST == ST - 1 || t == nt - 1) {
          __syncwarp();                              // the slot has been read
          slot ^= 1;
          phase ^= slot ^ 1;
          ++done;
          if (issued < total) fetch();
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint2 u0 = w[b][0], u1 = w[b][1];
          uint32_t a[16];
          a[0] = dc_pair<0>(u0.x, lanebyte);  a[1] = dc_pair<0>(u1.x, lanebyte);
          a[2] = dc_pair<1>(u0.x, lanebyte);  a[3] = dc_pair<1>(u1.x, lanebyte);
          a[4] = dc_pair<2>(u0.x, lanebyte);  a[5] = dc_pair<2>(u1.x, lanebyte);
          a[6] = dc_pair<3>(u0.x, lanebyte);  a[7] = dc_pair<3>(u1.x, lanebyte);
          a[8] = dc_pair<0>(u0.y, lanebyte);  a[9] = dc_pair<0>(u1.y, lanebyte);
          a[10] = dc_pair<1>(u0.y, lanebyte); a[11] = dc_pair<1>(u1.y, lanebyte);
          a[12] = dc_pair<2>(u0.y, lanebyte); a[13] = dc_pair<2>(u1.y, lanebyte);
          a[14] = dc_pair<3>(u0.y, lanebyte); a[15] = dc_pair<3>(u1.y, lanebyte);
          const float s0 = __uint_as_float(dc_word(f0, b)), s1 = __uint_as_float(dc_word(f1, b));
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            float d[4] = {};
#pragma unroll
            for (int q = 0; q < 4; ++q)
              c1_mma(d, a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3], dc_word(x[b][m][q >> 1], 2 * (q & 1)),
                     dc_word(x[b][m][q >> 1], 2 * (q & 1) + 1));
            acc[t][m][0] = fmaf(s0, d[0], acc[t][m][0]);
            acc[t][m][1] = fmaf(s0, d[1], acc[t][m][1]);
            acc[t][m][2] = fmaf(s1, d[2], acc[t][m][2]);
            acc[t][m][3] = fmaf(s1, d[3], acc[t][m][3]);
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kC4Tiles; ++t)
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        const uint32_t to = red + static_cast<uint32_t>(warp) * C::SUM_BYTES + 4u * ((t * 16 + gr) * TT + 8 * m + 2 * j);
        cl_sts2(to, acc[t][m][0], acc[t][m][1]);
        cl_sts2(to + 4u * 8 * TT, acc[t][m][2], acc[t][m][3]);
      }
    __syncthreads();
    auto mine = [&](int e) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) sum += cl_lds(red + static_cast<uint32_t>(w) * C::SUM_BYTES + 4u * e);
      return sum;
    };
    if constexpr (PAIR) {                            // one tile: one pass
      if (rank == 1)
        for (int e = threadIdx.x; e < nt * 16 * TT; e += blockDim.x) cl_st_peer(base + 4u * e, 0, mine(e));
      cl_cluster_sync();
    }
    if (rank == 0) {
      for (int e = threadIdx.x; e < nt * 16 * TT; e += blockDim.x) {
        float sum = mine(e);
        if constexpr (PAIR) sum += cl_lds(base + 4u * e);
        const int row = t0 * 16 + e / TT, t = e % TT;
        if (row < p.N && t < T) p.Y[static_cast<int64_t>(tok0 + t) * p.N + row] = __float2bfloat16_rn(sum * p.unscale);
      }
    }
    __syncthreads();
  }
  for (; done < issued; ++done) {                    // after a wait that gave up: this warp's copies in flight
    mbar_wait_short_addr(bars + 8 * slot, phase);
    slot ^= 1;
    phase ^= slot ^ 1;
  }
}
template <int NT, bool VEC>
__global__ void __launch_bounds__(C4<NT>::WARPS * 32, 1)
    codebook_linear4_kernel(const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmS,
                            const __grid_constant__ ClParams p, const __grid_constant__ CodebookArg cb) {
  codebook_linear4<NT, VEC, false>(tmC, tmS, p, cb);
}
template <int NT, bool VEC>
__global__ void __launch_bounds__(C4<NT>::WARPS * 32, 1) __cluster_dims__(2, 1, 1)
    codebook_linear4_pair_kernel(const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmS,
                                 const __grid_constant__ ClParams p, const __grid_constant__ CodebookArg cb) {
  codebook_linear4<NT, VEC, true>(tmC, tmS, p, cb);
}

}  // namespace qnf4
