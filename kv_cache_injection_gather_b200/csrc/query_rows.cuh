// Head rows of the query side: RMS norm and RoPE rotation of queries and
// keys, and the append of keys and values to the paged cache.
//
// Per row x of D elements at position p:
//   n_d = x_d * w_d * rsqrt(mean(x^2) + eps)          (or x_d without norm)
//   (a, b) -> (a cos - b sin, b cos + a sin)          per pair i, angle p f_i
// in fp32 from bf16, one rounding to bf16 at the end.  The work is a copy with
// a few operations an element: HBM bandwidth bounds long batches, the latency
// of a launch and of two dependent loads short ones.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace isq {

enum : int32_t {
  kErrInvalidArg = -1,
  kErrPosition = -3,
  kErrBadBlock = -4,
  kErrTimeout = -8,
};

struct Status {
  int32_t code;
  int32_t pad;
  long long detail;
};

// The first error is kept.
__device__ __forceinline__ void record(Status* st, int32_t code, long long detail) {
  if (atomicCAS(&st->code, 0, code) == 0) st->detail = detail;
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two fp32 values to two bf16 (round to nearest even), `lo` in the low half.
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Rows of one role: element (t, h, d) at data[t * ts + h * hs + d].
struct Rows {
  uint16_t* data;
  int64_t ts, hs;
};

struct RowArgs {
  const int32_t* positions;
  const int64_t* slots;        // append; nullptr: k goes to k_out, no v
  int32_t nq, nk, nv;          // heads of each role (0: absent)
  Rows q, q_out, k, k_out, v;
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  float eps;
  const double* turns;         // [D/2] RoPE frequencies over 2 pi
  // paged cache, at the layer
  uint16_t* k_cache;
  uint16_t* v_cache;
  int64_t block_stride, token_stride, head_stride;
  int64_t num_slots;
  int32_t block_size;
  Status* st;
};

// RoPE frequencies over 2 pi, fp64: theta^(-2i/D) with the Llama-3.1
// wavelength-band rule where scaling is 1 (wavelength 2 pi / f below
// orig/high: kept; above orig/low: divided by factor; blended between).
__global__ void turns_kernel(double* out, int D, double theta, int scaling, double factor, double low,
                             double high, double orig) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= D / 2) return;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  double f = pow(theta, -2.0 * double(i) / double(D));
  if (scaling == 1) {
    const double wave = kTwoPi / f;
    if (wave > orig / low) {
      f /= factor;
    } else if (wave >= orig / high) {
      const double w = (orig / wave - low) / (high - low);
      f = (1.0 - w) * (f / factor) + w * f;
    }
  }
  out[i] = f / kTwoPi;
}

// cos and sin of position * frequency.  The angle in turns is reduced by its
// whole part inside one fused multiply-add in fp64 (the product is not
// rounded before the subtraction), so the fraction is good to 2^-53 of the
// turns; sincospi then works on a number in [-1, 1] in fp32, accurate to
// about an fp32 unit in the last place for small results too.
__device__ __forceinline__ float2 cos_sin(int32_t position, double turns) {
  const double p = double(position);
  const double whole = rint(p * turns);
  const float x = float(2.0 * fma(p, turns, -whole));
  float s, c;
  sincospif(x, &s, &c);
  return make_float2(c, s);
}

// Plain (coherent) 16-byte accesses: an output may be its own input.
__device__ __forceinline__ uint4 ld16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void st16(uint16_t* p, const uint4& v) { *reinterpret_cast<uint4*>(p) = v; }

__device__ __forceinline__ void unpack(const uint4& u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = lo_f(w[i]);
    x[2 * i + 1] = hi_f(w[i]);
  }
}

__device__ __forceinline__ uint4 pack(const float* x) {
  return make_uint4(to_bf16x2(x[0], x[1]), to_bf16x2(x[2], x[3]), to_bf16x2(x[4], x[5]), to_bf16x2(x[6], x[7]));
}

// One CTA per token.  D/16 threads share a row; a thread holds the 16-byte
// vectors c and c + D/16 of it, so that both members of a rotate-half pair
// (i, i + D/2), and of an adjacent pair (2i, 2i + 1), are its own: no
// exchange but the norm's sum over the row's threads.  The token's cos and
// sin are computed once, by the first D/2 threads, while the first rows'
// loads are in flight, and laid out so that the row's threads read 16 bytes
// each from different banks.
constexpr int kRowThreads = 512;  // most threads of a CTA

template <int D, int STYLE>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ RowArgs a) {
  constexpr int TPR = D / 16;          // threads of a row
  const int NT = blockDim.x;           // a multiple of 32
  const int RPP = NT / TPR;            // rows of a pass
  // 8 (cos, sin) pairs per thread of a row, as 4 float4: [j][c]
  __shared__ float4 cs[4][TPR];
  const int tid = threadIdx.x;
  const int c = tid % TPR;
  const int64_t t = blockIdx.x;
  const int32_t pos = a.positions[t];
  if (pos < 0) return;
  int64_t slot = -1;
  if (a.slots != nullptr) {
    slot = a.slots[t];
    if (slot < -1 || slot >= a.num_slots) {
      if (tid == 0) record(a.st, kErrBadBlock, t);
      slot = -1;
    }
  }
  const int64_t block = slot < 0 ? 0 : slot / a.block_size;
  const int64_t cache_at =
      slot < 0 ? -1 : block * a.block_stride + (slot - block * a.block_size) * a.token_stride;
  const int rows = a.nq + a.nk + a.nv;

  auto source = [&](int w) -> const uint16_t* {
    if (w < a.nq) return a.q.data + t * a.q.ts + w * a.q.hs;
    w -= a.nq;
    if (w < a.nk) return a.k.data + t * a.k.ts + w * a.k.hs;
    return a.v.data + t * a.v.ts + (w - a.nk) * a.v.hs;
  };
  auto target = [&](int w) -> uint16_t* {
    if (w < a.nq) return a.q_out.data + t * a.q_out.ts + w * a.q_out.hs;
    w -= a.nq;
    if (w < a.nk) {
      if (a.slots == nullptr) return a.k_out.data + t * a.k_out.ts + w * a.k_out.hs;
      return cache_at < 0 ? nullptr : a.k_cache + cache_at + w * a.head_stride;
    }
    return cache_at < 0 ? nullptr : a.v_cache + cache_at + (w - a.nk) * a.head_stride;
  };

  uint4 u0, u1;
  int w = tid / TPR;
  if (w < rows) {
    const uint16_t* p = source(w);
    u0 = ld16(p + c * 8);
    u1 = ld16(p + D / 2 + c * 8);
  }
  for (int i = tid; i < D / 2; i += NT) {
    // Rotate-half: thread i / 8 owns pairs 8c .. 8c + 7.  Adjacent: vector c
    // holds pairs 4c .. 4c + 3 (its first four), vector c + D/16 the pairs
    // D/4 + 4c .. (its last four).
    const int owner = STYLE == 0 ? i / 8 : (i % (D / 4)) / 4;
    const int at = STYLE == 0 ? i % 8 : (i % (D / 4)) % 4 + (i >= D / 4 ? 4 : 0);
    reinterpret_cast<float2*>(&cs[at / 2][owner])[at % 2] = cos_sin(pos, a.turns[i]);
  }
  __syncthreads();

  // Whole warps stay in the loop: the norm's sum is a shuffle over the row.
  for (int first = 0; first < rows; first += RPP) {
    w = first + tid / TPR;
    const bool live = w < rows;
    if (first > 0 && live) {
      const uint16_t* p = source(w);
      u0 = ld16(p + c * 8);
      u1 = ld16(p + D / 2 + c * 8);
    }
    uint16_t* out = live ? target(w) : nullptr;
    if (w < a.nq + a.nk) {
      float x[16];
      unpack(u0, x);
      unpack(u1, x + 8);
      const uint16_t* weight = w < a.nq ? a.q_weight : a.k_weight;
      // rows of a role with and without norm can meet in one warp: the sum
      // is taken by all of them
      float sq = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) sq = fmaf(x[i], x[i], sq);
      const unsigned group = TPR == 32 ? 0xffffffffu : ((1u << TPR) - 1u) << ((tid & 31) / TPR * TPR);
#pragma unroll
      for (int m = TPR / 2; m > 0; m /= 2) sq += __shfl_xor_sync(group, sq, m);
      if (weight != nullptr) {
        const float r = rsqrtf(sq * (1.0f / D) + a.eps);
        float g[16];
        unpack(ld16(weight + c * 8), g);
        unpack(ld16(weight + D / 2 + c * 8), g + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] * r * g[i];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 v = cs[j][c];
        const float co[2] = {v.x, v.z}, si[2] = {v.y, v.w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = 2 * j + e;
          const int ia = STYLE == 0 ? i : 2 * i;
          const int ib = STYLE == 0 ? i + 8 : 2 * i + 1;
          const float xa = x[ia], xb = x[ib];
          x[ia] = xa * co[e] - xb * si[e];
          x[ib] = xb * co[e] + xa * si[e];
        }
      }
      u0 = pack(x);
      u1 = pack(x + 8);
    }
    if (out != nullptr) {
      st16(out + c * 8, u0);
      st16(out + D / 2 + c * 8, u1);
    }
  }
}

}  // namespace isq
