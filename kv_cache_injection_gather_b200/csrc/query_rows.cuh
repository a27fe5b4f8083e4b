// Head rows of the query side: RMS norm and RoPE rotation of queries and
// keys, and the append of keys and values to the paged cache.
//
// Per row x of D elements at position p:
//   n_d = x_d * w_d * rsqrt(mean(x^2) + eps)          (or x_d without norm)
//   (a, b) -> (a cos - b sin, b cos + a sin)          per pair i, angle p f_i
// in fp32 from bf16, one rounding to bf16 at the end.  The work is a copy with
// a few operations an element: HBM bandwidth bounds long batches, the latency
// of a launch and of two dependent loads short ones.  Measured on B200 (32
// query and 8 KV heads of 128): append of 16384 tokens 63.5 us, 0.98 of the copy
// bandwidth; rotate of 16384 tokens with norm 60 us, 0.87 (128 registers a
// thread, as the launch bound of 512 threads leaves them, make 16 warps an SM,
// the norm's shuffles stand between load and store, and the kernels with a norm
// spill 48 to 64 bytes a thread under that bound); up to 300 tokens 4.2 us.
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

// The first error since the last one was taken, in one word so that its code
// and detail arrive and leave together: code in the upper half (0: none),
// detail in the lower.
struct Status {
  unsigned long long first;
  unsigned long long taken;  // for the host
};

__device__ __forceinline__ void record(Status* st, int32_t code, int32_t detail) {
  atomicCAS(&st->first, 0ull, (static_cast<unsigned long long>(static_cast<uint32_t>(code)) << 32) | uint32_t(detail));
}

// Takes the error in the order of the stream that it is launched on.
__global__ void take_status_kernel(Status* st) { st->taken = atomicExch(&st->first, 0ull); }

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

// Two fp32 values in one 64-bit register, for the packed multiply and fused
// multiply-add.
using Two = uint64_t;
__device__ __forceinline__ Two two(float x, float y) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 both(Two v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Two from_bf16x2(uint32_t w) { return two(lo_f(w), hi_f(w)); }
__device__ __forceinline__ uint32_t to_bf16x2(Two v) {
  const float2 f = both(v);
  return to_bf16x2(f.x, f.y);
}
__device__ __forceinline__ Two swapped(Two v) {
  const float2 f = both(v);
  return two(f.y, f.x);
}
constexpr uint32_t kOnes = 0x3f803f80u;  // two bf16 ones

struct Vecs {
  uint4 lo, hi;  // the 16-byte vectors c and c + D/16 of a row
};
template <int D>
__device__ __forceinline__ Vecs load_row(const uint16_t* p) {
  return {ld16(p), ld16(p + D / 2)};
}
template <int D>
__device__ __forceinline__ void store_row(uint16_t* p, const Vecs& v) {
  st16(p, v.lo);
  st16(p + D / 2, v.hi);
}

// A thread's share of a rotation: two pairs a step, 4 steps.  With `x` the
// step's two words (rotate-half: elements 2j, 2j + 1 of both vectors; adjacent:
// words 2j and 2j + 1 of the 8), the results are x0 p[j][0] + other p[j][1] and
// x1 p[j][2] + other p[j][3], where `other` is the other word (rotate-half) or
// the word itself with its halves exchanged (adjacent).
struct Rotation {
  Two p[4][4];
};
template <int STYLE>
__device__ __forceinline__ void set_rotation(Rotation& r, const float4* cs, int step, const Vecs& g) {
  const uint32_t g0[4] = {g.lo.x, g.lo.y, g.lo.z, g.lo.w}, g1[4] = {g.hi.x, g.hi.y, g.hi.z, g.hi.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 v = cs[j * step];  // cos, cos, sin, sin of pairs 2j, 2j + 1 of this thread
    if constexpr (STYLE == 0) {
      const Two co = two(v.x, v.y), si = two(v.z, v.w), wa = from_bf16x2(g0[j]), wb = from_bf16x2(g1[j]);
      r.p[j][0] = mul(co, wa);
      r.p[j][1] = mul(two(-v.z, -v.w), wb);
      r.p[j][2] = mul(co, wb);
      r.p[j][3] = mul(si, wa);
    } else {
      const Two wa = from_bf16x2(j < 2 ? g0[2 * j] : g1[2 * j - 4]), wb = from_bf16x2(j < 2 ? g0[2 * j + 1] : g1[2 * j - 3]);
      r.p[j][0] = mul(two(v.x, v.x), wa);
      r.p[j][1] = mul(two(-v.z, v.z), swapped(wa));
      r.p[j][2] = mul(two(v.y, v.y), wb);
      r.p[j][3] = mul(two(-v.w, v.w), swapped(wb));
    }
  }
}

// Norm (with eps, over the row's threads) and rotation of a row.
template <int D, int STYLE, bool NORM>
__device__ __forceinline__ Vecs turn_row(const Vecs& in, const Rotation& rot, bool normed, float eps) {
  constexpr int TPR = D / 16;
  const uint32_t u[8] = {in.lo.x, in.lo.y, in.lo.z, in.lo.w, in.hi.x, in.hi.y, in.hi.z, in.hi.w};
  Two x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = from_bf16x2(u[i]);
  if (NORM && normed) {
    Two sq = mul(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) sq = fma2(x[i], x[i], sq);
    const float2 f = both(sq);
    float sum = f.x + f.y;
    const unsigned group = ((1u << TPR) - 1u) << ((threadIdx.x & 31) / TPR * TPR);
#pragma unroll
    for (int m = TPR / 2; m > 0; m /= 2) sum += __shfl_xor_sync(group, sum, m);
    const float r = rsqrtf(sum * (1.0f / D) + eps);
    const Two rr = two(r, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = mul(x[i], rr);
  }
  uint32_t y[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i0 = STYLE == 0 ? j : 2 * j, i1 = STYLE == 0 ? j + 4 : 2 * j + 1;
    const Two o0 = STYLE == 0 ? x[i1] : swapped(x[i0]), o1 = STYLE == 0 ? x[i0] : swapped(x[i1]);
    y[i0] = to_bf16x2(fma2(x[i0], rot.p[j][0], mul(o0, rot.p[j][1])));
    y[i1] = to_bf16x2(fma2(x[i1], rot.p[j][2], mul(o1, rot.p[j][3])));
  }
  return {make_uint4(y[0], y[1], y[2], y[3]), make_uint4(y[4], y[5], y[6], y[7])};
}

// One CTA per token.  D/16 threads share a row; a thread holds the 16-byte
// vectors c and c + D/16 of it, so that both members of a rotate-half pair
// (i, i + D/2), and of an adjacent pair (2i, 2i + 1), are its own: no exchange
// but the norm's sum over the row's threads.  Its 8 pairs' cos and sin (times
// the norm's weights) are the same for every row that it takes: they stay in
// registers.  They are computed once per token by the first D/2 threads, while
// the first rows of every role are on their way.
constexpr int kRowThreads = 512;  // most threads of a CTA
constexpr int kQueriesAhead = 4;  // query rows of a thread in flight (2: 63 us for 16384 tokens, 4: 60)

template <int D, int STYLE, bool NORM>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ RowArgs a) {
  constexpr int TPR = D / 16;          // threads of a row
  const int NT = blockDim.x;           // a multiple of 32
  const int RPP = NT / TPR;            // rows of a pass
  __shared__ float4 s_cs[4][TPR];      // see set_rotation; by thread of a row
  const int tid = threadIdx.x;
  const int c = tid % TPR, w0 = tid / TPR;
  const int64_t t = blockIdx.x;
  const bool append = a.slots != nullptr;

  const uint16_t* q_in = a.q.data + t * a.q.ts + w0 * a.q.hs + c * 8;
  const uint16_t* k_in = a.k.data + t * a.k.ts + w0 * a.k.hs + c * 8;
  const uint16_t* v_in = a.v.data + t * a.v.ts + w0 * a.v.hs + c * 8;
  const int64_t q_step = RPP * a.q.hs, k_step = RPP * a.k.hs, v_step = RPP * a.v.hs;
  Vecs q[kQueriesAhead], k, v;
#pragma unroll
  for (int i = 0; i < kQueriesAhead; ++i)
    if (w0 + i * RPP < a.nq) q[i] = load_row<D>(q_in + i * q_step);
  if (w0 < a.nk) k = load_row<D>(k_in);
  if (w0 < a.nv) v = load_row<D>(v_in);
  const int32_t pos = a.positions[t];
  int64_t slot = append ? a.slots[t] : -1;
  if (pos < 0) return;
  for (int i = tid; i < D / 2; i += NT) {
    // Rotate-half: thread i / 8 owns pairs 8c .. 8c + 7.  Adjacent: vector c
    // holds pairs 4c .. 4c + 3 (its first four), vector c + D/16 the pairs
    // D/4 + 4c .. (its last four).
    const int owner = STYLE == 0 ? i / 8 : (i % (D / 4)) / 4;
    const int at = STYLE == 0 ? i % 8 : (i % (D / 4)) % 4 + (i >= D / 4 ? 4 : 0);
    const float2 v2 = cos_sin(pos, a.turns[i]);
    float* to = reinterpret_cast<float*>(&s_cs[at / 2][owner]) + at % 2;
    to[0] = v2.x;
    to[2] = v2.y;
  }
  if (append && (slot < -1 || slot >= a.num_slots)) {
    if (tid == 0) record(a.st, kErrBadBlock, int32_t(t));
    slot = -1;
  }
  __syncthreads();

  Rotation rot;
  auto set_role = [&](const uint16_t* weight) {
    Vecs g = {make_uint4(kOnes, kOnes, kOnes, kOnes), make_uint4(kOnes, kOnes, kOnes, kOnes)};
    if (NORM && weight != nullptr) g = load_row<D>(weight + c * 8);
    set_rotation<STYLE>(rot, &s_cs[0][c], TPR, g);
  };
  set_role(a.q_weight);
  {
    uint16_t* out = a.q_out.data + t * a.q_out.ts + w0 * a.q_out.hs + c * 8;
    const int64_t out_step = RPP * a.q_out.hs;
    for (int w = w0; w < a.nq;) {  // a row's threads stay together
#pragma unroll
      for (int i = 0; i < kQueriesAhead; ++i) {
        if (w >= a.nq) break;
        const Vecs y = turn_row<D, STYLE, NORM>(q[i], rot, a.q_weight != nullptr, a.eps);
        if (w + kQueriesAhead * RPP < a.nq) q[i] = load_row<D>(q_in + (i + kQueriesAhead) * q_step);
        store_row<D>(out, y);
        out += out_step;
        w += RPP;
      }
      q_in += kQueriesAhead * q_step;
    }
  }
  uint16_t* k_out = a.k_out.data + t * a.k_out.ts;
  int64_t out_hs = a.k_out.hs, cache_at = 0;
  if (append) {
    if (slot < 0) return;  // not stored
    const int64_t block = slot / a.block_size;
    cache_at = block * a.block_stride + (slot - block * a.block_size) * a.token_stride;
    k_out = a.k_cache + cache_at;
    out_hs = a.head_stride;
  }
  if (NORM) set_role(a.k_weight);
  k_out += w0 * out_hs + c * 8;
  for (int w = w0; w < a.nk; w += RPP) {
    store_row<D>(k_out, turn_row<D, STYLE, NORM>(k, rot, a.k_weight != nullptr, a.eps));
    k_in += k_step;
    k_out += RPP * out_hs;
    if (w + RPP < a.nk) k = load_row<D>(k_in);
  }
  uint16_t* v_out = a.v_cache + cache_at + w0 * out_hs + c * 8;
  for (int w = w0; w < a.nv; w += RPP) {
    store_row<D>(v_out, v);
    v_in += v_step;
    v_out += RPP * out_hs;
    if (w + RPP < a.nv) v = load_row<D>(v_in);
  }
}

}  // namespace isq
