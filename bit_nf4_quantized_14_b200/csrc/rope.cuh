// Rotary positions: every pair (a, b) of the first rotary_dim features of a head is turned by the angle
// p * theta_i of its token's position p, and scaled by m:
//     a' = m (a cos - b sin),   b' = m (b cos + a sin);
// the pairs are features (i, i + R/2) (half layout) or (2i, 2i + 1) (interleaved). The rest of the head
// passes through. The gradient of a rotation is the rotation by -p theta, so `inverse` is the backward.
//
// What bounds it: HBM, one read and one write of every element (3 FLOP per element). The angles are shared
// by all heads of a token, so a CTA first forms the sines and cosines of its tokens in shared memory, one
// per thread, and then every thread keeps one chunk of pairs (its sines and cosines in registers) and walks
// over the heads of both tensors, one 16-byte access per operand where sizes and strides allow it.
//
// Angles: p * theta / (2 pi) is formed in fp64, where even p = 2^31 leaves 2^-22 of a turn; its fraction of a
// turn, in [-1/2, 1/2], is rounded once to fp32 and goes to sincospif. Everything else is fp32, rounded once
// to the element type at the end.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace qnf4 {

constexpr int kRopeMaxPairs = 256;     // rotary_dim <= 512
constexpr int kRopeThreads = 256;      // units of one head x head slots, at most (more only when one head has more)
constexpr int kRopeMaxTensors = 2;

struct RopeSide {                      // one tensor: heads x head_dim per token; strides in elements
  const void* in;
  void* out;
  int64_t in_b, in_t, in_h, out_b, out_t, out_h;
};
struct RopeParams {
  RopeSide x[kRopeMaxTensors];
  int heads0, heads;                   // heads of x[0], and of all tensors together
  int64_t T, tokens;                   // tokens per batch row, and in all
  int rotary_dim, head_dim;
  int units, tail;                     // chunks of pairs per head, and chunks copied per head
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

// VE: elements of one access, aligned to AL elements (AL < VE only for interleaved pairs at odd strides). Half
// layout: a unit is VE features of the first half and the VE that pair with them; interleaved: VE / 2 pairs side
// by side. TOK: tokens per CTA.
template <typename T, int VE, int AL, bool HALF, int TOK>
__global__ void rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int PAIRS = HALF ? VE : VE / 2;
  using Vec = RopeVec<T, VE, AL>;
  extern __shared__ float rope_sm[];                 // [TOK][R/2] cosines, then sines
  const int half = p.rotary_dim / 2;
  float* cs = rope_sm;
  float* sn = rope_sm + TOK * half;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * TOK;
  const int ntok = static_cast<int>(min(static_cast<int64_t>(TOK), p.tokens - tok0));

  for (int e = threadIdx.x; e < ntok * half; e += blockDim.x) {
    const int i = e / half, pair = e - i * half;
    const int64_t tok = tok0 + i, b = tok / p.T, t = tok - b * p.T;
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
    cs[e] = c * p.mscale;
    sn[e] = (p.inverse ? -s : s) * p.mscale;
  }
  __syncthreads();

  const int per_head = p.units + p.tail;
  const int u = threadIdx.x % per_head, slot = threadIdx.x / per_head;
  const int h_end = min(p.heads, static_cast<int>(blockIdx.y + 1) * p.heads_per_cta);
  for (int i = 0; i < ntok; ++i) {
    const int64_t tok = tok0 + i, b = tok / p.T, t = tok - b * p.T;
    float c[PAIRS], s[PAIRS];
    if (u < p.units) {
#pragma unroll
      for (int k = 0; k < PAIRS; ++k) {
        c[k] = cs[i * half + u * PAIRS + k];
        s[k] = sn[i * half + u * PAIRS + k];
      }
    }
#pragma unroll 2
    for (int h = blockIdx.y * p.heads_per_cta + slot; h < h_end; h += p.slots) {
      const bool second = h >= p.heads0;
      const RopeSide& x = p.x[second ? 1 : 0];
      const int hh = second ? h - p.heads0 : h;
      const T* in = static_cast<const T*>(x.in) + b * x.in_b + t * x.in_t + hh * x.in_h;
      T* out = static_cast<T*>(x.out) + b * x.out_b + t * x.out_t + hh * x.out_h;
      if (u >= p.units) {                            // features behind the rotated part
        const int f = p.rotary_dim + (u - p.units) * VE;
        if (f + VE <= p.head_dim) *reinterpret_cast<Vec*>(out + f) = *reinterpret_cast<const Vec*>(in + f);
        else
          for (int k = f; k < p.head_dim; ++k) out[k] = in[k];
      } else if constexpr (HALF) {
        const int f = u * VE;
        Vec lo = *reinterpret_cast<const Vec*>(in + f), hi = *reinterpret_cast<const Vec*>(in + f + half);
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          const float a = rope_load(lo.v[k]), d = rope_load(hi.v[k]);
          lo.v[k] = rope_store<T>(a * c[k] - d * s[k]);
          hi.v[k] = rope_store<T>(d * c[k] + a * s[k]);
        }
        *reinterpret_cast<Vec*>(out + f) = lo;
        *reinterpret_cast<Vec*>(out + f + half) = hi;
      } else {
        const int f = u * VE;
        Vec w = *reinterpret_cast<const Vec*>(in + f);
#pragma unroll
        for (int k = 0; k < PAIRS; ++k) {
          const float a = rope_load(w.v[2 * k]), d = rope_load(w.v[2 * k + 1]);
          w.v[2 * k] = rope_store<T>(a * c[k] - d * s[k]);
          w.v[2 * k + 1] = rope_store<T>(d * c[k] + a * s[k]);
        }
        *reinterpret_cast<Vec*>(out + f) = w;
      }
    }
  }
}

}  // namespace qnf4
