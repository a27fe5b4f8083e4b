// Attention over the paged cache for many query rows per KV head (prompts,
// the query tokens of a request): the products bound it, so they run on the
// fifth-generation tensor cores (tcgen05) with the scores and the output sum
// in tensor memory.
//
// A CTA takes a unit of up to 256 rows -- (token, head) pairs of one request
// that share a KV head -- and walks its keys in tiles of 128:
//
//   S = Q K^T (128 x 128, fp32 in tensor memory)
//   P = exp2(scale S - m), in bf16, over S in tensor memory
//   O += P V
//
// Two streams keep the tensor cores busy while a stream's softmax runs.  A
// unit of more than 128 rows gives each stream 128 rows and every key tile; a
// smaller one gives both streams the same rows and every other key tile, and
// their sums are joined at the end.
//
// Warps 0-3 and 4-7 do the streams' softmax, one row a thread; warps 8 on
// gather keys and values from the cache's blocks into a ring of 128-key tiles
// (TMA boxes of a block's tokens, in the 128-byte swizzle that the products
// read); the last two issue a stream's products each, from one thread.
// mbarriers join them.  Every wait is bounded: a thread that gives up sets a
// flag that all see, the CTA drains, frees its tensor memory and records
// IS_ERR_TIMEOUT.
//
// A tile goes through a stream in halves of 64 keys: while one half's softmax
// runs, the products of the other are under way -- its values', and behind them
// the next tile's scores.
//
// Measured on B200 (32 query and 8 KV heads of 128): two causal prompts of
// 4096 tokens 280-315 us (850-960 TFLOP/s, 0.51-0.58 of the burst bf16 GEMM;
// the spread is the card's power limit), 100 requests of 16-64 queries over
// 3300-5000 keys 382 us (690 TFLOP/s of what is not masked or padded) on a cool
// card, 435 (610) on one that is warm from other products; with a tile as one
// piece 303-328 and 412 us.  A tile of both streams takes 3400
// cycles.  Its halves alternate between softmax (maximum 300, exponentials
// 1100, 770 of which the special-function units take for both streams) and
// products (both streams' 1300, as scores of 64 keys read more shared memory
// than they compute on, and 350 from the last probability to the first
// product and from the last product to the next maximum): the two phases are
// equally long, and neither waits for the other alone.  Products in strict turns,
// from two threads or one, shorten the softmax to 1050 but idle between turns:
// the same 3400.  A unit's start costs 8200 cycles (its queries arrive at 6600),
// its end 6600 and the next CTA 1300, of some 60 000 for 4096 keys.
#pragma once

#include "attend_common.cuh"

namespace isq {

constexpr int kStreamRows = 128;
constexpr int kUnitRows = 2 * kStreamRows;

template <int D>
struct TilesShape {
  static constexpr int kSlotBytes = kTileKeys * D * 2;   // one K or V tile
  static constexpr int kSlots = D == 128 ? 4 : 8;
  // By time: 100 requests of 16-64 queries with 4 gather warps 396 us, 2: 385, 1:
  // 476.  (Registers do not decide it: a thread uses 125 of the 168 that 12 warps
  // leave, and 14 warps would leave 144.)  One warp a stream issues its products: a wait costs a lone thread some 200
  // cycles of latency, and a tile has four.
  static constexpr int kGather = 2;
  static constexpr int kProductWarp = 8 + kGather;       // and the next
  static constexpr int kThreads = (8 + kGather + 2) * 32;
  static constexpr int kQBytes = kUnitRows * D * 2;
  // data, and up to 1 KB to align it
  static constexpr int kSmemBytes = kQBytes + kSlots * kSlotBytes + 1024;
};

// ---------------------------------------------------------------- the kernel

// Of 8 exponentials, those on the multiply-add units.  100 requests of 16-64
// queries, with 4 gather warps 0: 408 us, 1: 401, 2: 396, 3: 398; with 2 gather
// warps 1: 389, 2: 385, 3: 385.
constexpr int kPolynomial = 2;

struct Yes {
  static constexpr bool value = true;
};
struct No {
  static constexpr bool value = false;
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 2^x of two values up to 2^7 without the special-function unit: x = n + f with
// n whole and |f| <= 1/2, 2^f by a polynomial of degree 4 (the coefficients
// minimise the largest relative error on that interval, 2.6e-6 = 2^-18.5,
// found by reweighted least squares), times 2^n.  Below 2^-126 it stays there.
// Adding 1.5 * 2^23 leaves n in a sum's low bits.  A NaN stays one: it goes
// through the polynomial and the product (n added to the exponent's bits would
// make a NaN a large number).
__device__ __forceinline__ Two exp2_two(Two x) {
  const float2 in = both(x);
  float lo, hi;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(lo) : "f"(in.x), "f"(-126.f));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(hi) : "f"(in.y), "f"(-126.f));
  x = two(lo, hi);
  const Two round = two(12582912.f, 12582912.f), back = two(-12582912.f, -12582912.f), minus = two(-1.f, -1.f);
  const Two t = add2(x, round);
  const Two f = fma2(add2(t, back), minus, x);
  Two p = two(0.009570102207362652f, 0.009570102207362652f);
  p = fma2(p, f, two(0.05591785907745361f, 0.05591785907745361f));
  p = fma2(p, f, two(0.240247443318367f, 0.240247443318367f));
  p = fma2(p, f, two(0.6931217908859253f, 0.6931217908859253f));
  p = fma2(p, f, two(0.9999992847442627f, 0.9999992847442627f));
  const float2 n = both(t);  // bits of 2^n: n + 127 in the exponent
  return mul(p, two(__uint_as_float((__float_as_uint(n.x) << 23) + 0x3f800000u),
                    __uint_as_float((__float_as_uint(n.y) << 23) + 0x3f800000u)));
}

// The request that owns query token t: the last r with q_offsets[r] <= t.
__device__ __forceinline__ int32_t owner_of(const AttendArgs& a, int32_t t) {
  int32_t at = 0, n = a.num_requests;
  while (n > 1) {
    const int32_t half = n / 2;
    if (a.q_offsets[at + half] <= t) {
      at += half;
      n -= half;
    } else {
      n = half;
    }
  }
  return at;
}

// Token (of the request) and head (of the KV head's) of rows in steps.
struct RowWalk {
  int32_t token, g;
  int32_t group, step_token, step_g;
  __device__ __forceinline__ RowWalk(int32_t group_, int32_t row, int32_t step)
      : token(row / group_), g(row - token * group_), group(group_), step_token(step / group_),
        step_g(step - step_token * group_) {}
  __device__ __forceinline__ void step() {
    token += step_token;
    g += step_g;
    if (g >= group) {
      g -= group;
      ++token;
    }
  }
};

// SHARED: the units are 256 rows of all requests' query tokens, and their keys
// those of the shared prefix; otherwise rows and keys of one request.  Where
// a.part_o is set, split s of a unit's keys goes to part s of the work space;
// otherwise there is one split and it goes to the output.
template <int D, bool SHARED>
__global__ void __launch_bounds__(TilesShape<D>::kThreads, 1) attend_tiles_kernel(
    const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap k_map,
    const __grid_constant__ CUtensorMap v_map) {
  using S = TilesShape<D>;
  constexpr int CPR = D / 8, NS = S::kSlots;
  // P meets V rounded to bf16, as the tensor cores take both operands in one
  // type: an error of up to 2^-8 of sum p |v| beside the result's rounding.  For
  // a prefix (decode) the remainder of the rounding goes in as well, behind P in
  // the scores' columns, and P is good to 2^-16: 100 requests behind 4096 shared
  // tokens 168 -> 171 us, behind 16384 134 -> 140.  Where the products bound the
  // call it would cost a fifth (100 requests of 16-64 queries 381 -> 463 us, two
  // prompts of 4096 tokens 282-315 -> 330-366), so there it stays rounded.
  constexpr bool kRest = SHARED;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[NS], bar_empty[NS], bar_q, bar_s[2][2], bar_p[2][2], bar_o[2][2],
      bar_end[2], bar_edge;
  __shared__ uint32_t s_tmem;
  __shared__ int32_t s_failed, s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;

  let_next_start();
  // grid: (unit, KV head, split), and a CTA that checks the batch (in SHARED
  // the grid that follows does)
  const int32_t split = int32_t(blockIdx.x % a.splits);
  const int32_t h = int32_t(blockIdx.x / a.splits) % a.kv_heads;
  // (the last units first: with a causal mask they see the most keys)
  const int32_t unit = int32_t(a.units) - 1 - int32_t(blockIdx.x / a.splits) / a.kv_heads;
  if (!SHARED && blockIdx.x == gridDim.x - 1) {
    check_requests<S::kThreads>(a);
    return;
  }
  // what needs no metadata first, a barrier a thread
  if (tid < NS) {
    bar_init(&bar_full[tid], 1);
    bar_init(&bar_empty[tid], 2);
  } else if (tid >= 32 && tid < 34) {
    for (int i = 0; i < 2; ++i) {
      bar_init(&bar_s[tid - 32][i], 1);
      bar_init(&bar_p[tid - 32][i], kStreamRows);
      bar_init(&bar_o[tid - 32][i], 1);
    }
    bar_init(&bar_end[tid - 32], 1);
  } else if (tid == 64) {
    bar_init(&bar_q, 2 * kStreamRows);
    bar_init(&bar_edge, 1);
    s_failed = 0;
    s_bad = 0;
  } else if (tid == 96) {
    fetch_map(&k_map);
    fetch_map(&v_map);
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (warp == S::kProductWarp) tmem_alloc(&s_tmem, 512);
  int32_t r, tile;
  Request rq;
  if constexpr (SHARED) {
    r = -1;
    tile = unit;
    rq = {0, a.num_tokens, 0, 0};
  } else {
    find_unit<kUnitRows, S::kThreads>(a, unit, r, tile, rq);
    if (r < 0) {
      if (warp == S::kProductWarp) tmem_free(s_tmem, 512);
      return;
    }
  }

  const int32_t row0 = tile * kUnitRows;
  const int32_t rows = int32_t(min(int64_t(kUnitRows), int64_t(rq.n) * a.group - row0));
  auto token_of = [&](int row) { return (row0 + row) / a.group; };
  auto head_of = [&](int row) { return h * a.group + (row0 + row) % a.group; };
  // First key that a row does not see.
  auto limit_of = [&](int row) -> int32_t {
    if constexpr (!SHARED) return row_limit(a, rq, token_of(row));
    const int32_t t = token_of(row), o = owner_of(a, t);
    Request q;
    if (read_request(a, o, q) != 0 || t < q.tok0 || t >= q.tok0 + q.n) return 0;
    return row_limit(a, q, t - q.tok0);
  };
  // keys [lo, hi) of this CTA: whole tiles but the last
  const int32_t all = SHARED ? a.shared_len : limit_of(rows - 1);
  // (below 2^24 tiles, times up to 32 splits)
  const uint32_t all_tiles = (uint32_t(all) + kTileKeys - 1) / kTileKeys;
  const int32_t lo = int32_t(all_tiles * split / a.splits) * kTileKeys;
  const uint32_t last = all_tiles * (split + 1) / a.splits;
  const int32_t hi = last == all_tiles ? all : int32_t(last) * kTileKeys;
  const int32_t tiles = hi > lo ? (hi - lo + kTileKeys - 1) / kTileKeys : 0;
  const bool by_rows = rows > kStreamRows;
  // tiles of a stream: all of them, or every other
  auto tiles_of = [&](int st) { return by_rows ? tiles : (tiles - st + 1) / 2; };
  auto first_key_of = [&](int st, int32_t i) { return lo + (by_rows ? i : 2 * i + st) * kTileKeys; };

  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  unsigned char* ring = smem + S::kQBytes;

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;  // S0 | S1 (128 columns each) | O0 | O1 (D each)
  const uint32_t tmem_o = tmem + 256;
  constexpr int OC = 128;        // columns between O0 and O1
  constexpr int kRowStep = 2 * kStreamRows / CPR;  // rows that the softmax warps move at a time

  float m = neg_inf(), l = 0.f;  // softmax warps: of this thread's row
  int32_t lim = 0;

  if (warp >= 8 && warp < S::kProductWarp) {
    gather_tiles<D, NS, S::kGather>(a, &k_map, &v_map, warp - 8, r, h, lo, hi, tiles, ring, bar_full, bar_empty,
                                    &bar_edge, &s_failed, &s_bad);
  } else if (warp >= S::kProductWarp) {
    // ---------------- products of stream st
    const int st = warp - S::kProductWarp;
    const int32_t n = tiles_of(st);
    if (n > 0 && elect_one()) {
      const uint32_t ts = tmem + st * 128, to = tmem_o + st * OC;
      const uint32_t qa = smem_addr(smem) + (by_rows ? st * S::kSlotBytes : 0), ring_at = smem_addr(ring);
      const int step = by_rows ? 2 : 4;  // slots from a tile to the next; its values are in the next slot
      int slot = by_rows ? 0 : 2 * st, next = slot;
      uint32_t parity = 0, next_parity = 0;
      auto advance = [&] {
        next = slot + step;
        next_parity = parity;
        if (next >= NS) {
          next -= NS;
          next_parity ^= 1;
        }
      };
      auto free_slot = [&](int at) {  // two arrivals: both streams', or the one's that reads the tile
        tc_commit(&bar_empty[at]);
        if (!by_rows) tc_commit(&bar_empty[at]);
      };
      // scores of half a tile, its 64 keys from 64 * half on (descriptors count
      // in 16 bytes: a step along a tile is an addition)
      auto scores = [&](int at, int half) {
        tc_fence_after();
        const uint32_t ka = ring_at + at * S::kSlotBytes + half * (S::kSlotBytes / 2);
        const uint64_t qd = operand<D>(qa, 16), kd = operand<D>(ka, 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss(ts + half * 64, qd + (dims_at<D>(k) >> 4), kd + (dims_at<D>(k) >> 4),
                 product(kTileKeys / 2, false, false), k > 0);
        tc_commit(&bar_s[st][half]);
        if (half == 1) free_slot(at);
      };
      bool ok = bar_wait(&bar_q, 0, &s_failed) && bar_wait(&bar_full[slot], parity, &s_failed);
      if (ok) {
        scores(slot, 0);
        scores(slot, 1);
      }
      for (int32_t i = 0; i < n && ok; ++i) {
        advance();
        const bool more = i + 1 < n;
        // both tiles before the probabilities, which come last
        ok = bar_wait(&bar_full[slot + 1], parity, &s_failed) &&
             (!more || bar_wait(&bar_full[next], next_parity, &s_failed));
        const uint32_t va = ring_at + (slot + 1) * S::kSlotBytes;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          ok = ok && bar_wait(&bar_p[st][half], i & 1, &s_failed);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = operand<D>(va + half * (D * 128), kSlabStep);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(to, ts + half * 64 + k * 8, vd + k * (D * 32 / 16), product(D, false, true),
                   i > 0 || half > 0 || k > 0);
          if constexpr (kRest) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(to, ts + half * 64 + 32 + k * 8, vd + k * (D * 32 / 16), product(D, false, true), true);
          }
          tc_commit(&bar_o[st][half]);
          if (half == 1) free_slot(slot + 1);
          // (the next scores overwrite the probabilities that these products
          // read: products run in the order of their issue)
          if (more) scores(next, half);
        }
        if (!ok) break;
        slot = next;
        parity = next_parity;
      }
      tc_commit(&bar_end[st]);
      bar_wait(&bar_end[st], 0, nullptr);  // nothing in flight beyond this point
    }
    __syncwarp();
  } else {
    // ---------------- softmax of stream st, one row a thread
    {
      RowWalk at(a.group, row0 + tid / CPR, kRowStep);
      const int c = tid % CPR;
      for (int row = tid / CPR; row < (by_rows ? kUnitRows : kStreamRows); row += kRowStep) {
        const bool live = row < rows;
        const uint16_t* src = a.q.data;
        if (live) src += int64_t(rq.tok0 + at.token) * a.q.ts + (h * a.group + at.g) * a.q.hs + c * 8;
        cp_async16(smem_addr(smem + tile_at<D>(row, c)), src, live ? 16 : 0);
        at.step();
      }
      cp_async_commit();
      cp_async_wait<0>();
      proxy_fence();
      bar_arrive(&bar_q);
    }
    const int st = warp / 4, row = (tid & 127) + (by_rows ? st * kStreamRows : 0);
    lim = row < rows ? min(hi, limit_of(row)) : hi;
    const int32_t lim_min = __reduce_min_sync(0xffffffffu, lim);
    const uint32_t lanes = uint32_t(warp & 3) << 21;  // 32 lanes a warp
    const uint32_t ts = tmem + st * 128 + lanes, to = tmem_o + st * OC + lanes;
    const int32_t n = 2 * tiles_of(st);  // halves
    for (int32_t it = 0; it < n; ++it) {
      const int half = it & 1;
      // the whole warp goes on or stops: what follows is warp-wide
      if (!__all_sync(0xffffffffu, bar_wait(&bar_s[st][half], (it >> 1) & 1, &s_failed))) break;
      tc_fence_after();
      const int32_t j0 = first_key_of(st, it >> 1) + half * 64;
      const bool masked = j0 + 64 > lim_min;
      const int32_t seen = lim - j0;  // columns below are seen
      const uint32_t tp = ts + half * 64;
      uint32_t v[64];
      tmem_ld<64>(tp, v);
      tmem_wait_ld();
      if (masked) {
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (i >= seen) v[i] = 0xff800000u;
      }
      float tops[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) tops[i] = fmaxf(__uint_as_float(v[i]), __uint_as_float(v[i + 4]));
#pragma unroll
      for (int i = 8; i < 64; i += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) tops[e] = max3(tops[e], __uint_as_float(v[i + e]), __uint_as_float(v[i + 4 + e]));
      // (the scale is positive: the maximum's place is the same)
      const float top = max3(fmaxf(tops[0], tops[1]), tops[2], tops[3]) * a.scale_log2;
      // The reference m follows the maximum only when that has risen by more
      // than 2^8: smaller steps leave P below 2^8 and O as it is.  All rows
      // of a warp take part in a correction (factor 1 where none is needed).
      float shrink = 1.f;
      if (top > m + 8.f) {  // (-inf + 8 is -inf: the first seen key counts)
        shrink = exp2_fast(m - top);
        m = top;
      }
      if (it > 0 && __any_sync(0xffffffffu, shrink != 1.f)) {
        l *= shrink;
        // the products with V up to the half before (those before it are done:
        // this half's scores were issued behind them)
        if (!__all_sync(0xffffffffu, bar_wait(&bar_o[st][half ^ 1], ((it - 1) >> 1) & 1, &s_failed))) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t o[16];
          tmem_ld<16>(to + c * 16, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * shrink);
          tmem_st<16>(to + c * 16, o);
        }
      }
      const float ref = m == neg_inf() ? 0.f : m;
      const Two scale2 = two(a.scale_log2, a.scale_log2), ref2 = two(-ref, -ref);
      Two sum2 = 0;
      // P, two keys at a time, over the scores (which are all read).  A share
      // of the exponentials is computed on the multiply-add units, as the
      // special-function unit's 16 a cycle are what a tile waits for; none where
      // keys are masked, or a row has no score above -inf yet (the polynomial
      // ends at 2^-126, and these have to be 0 exactly).
      auto probabilities = [&](auto plain) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t p[16];
          [[maybe_unused]] uint32_t rest[16];  // kRest: what the rounding left out (exact)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int at = c * 32 + 2 * i;
            const Two x = fma2(two(__uint_as_float(v[at]), __uint_as_float(v[at + 1])), scale2, ref2);
            Two e;
            if (!decltype(plain)::value && i % 8 < kPolynomial) {
              e = exp2_two(x);
            } else {
              const float2 f = both(x);
              e = two(exp2_fast(f.x), exp2_fast(f.y));
            }
            sum2 = add2(sum2, e);
            p[i] = to_bf16x2(e);
            if constexpr (kRest) rest[i] = to_bf16x2(fma2(from_bf16x2(p[i]), two(-1.f, -1.f), e));
          }
          tmem_st16(tp + c * 16, p);
          if constexpr (kRest) tmem_st16(tp + 32 + c * 16, rest);
        }
        tmem_wait_st();
        tc_fence_before();
        bar_arrive(&bar_p[st][half]);
      };
      if (masked || __any_sync(0xffffffffu, m == neg_inf())) probabilities(Yes());
      else probabilities(No());
      const float2 sums = both(sum2);
      l += sums.x + sums.y;
    }
  }

  // ---------------- output
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const bool failed = s_failed != 0;
  if (failed && tid == 0) record(a.st, kErrTimeout, unit);
  if (!failed && warp < 8) {
    const int st = warp / 4;
    const int rr = tid & 127;
    const uint32_t to = tmem_o + st * OC + (uint32_t(warp & 3) << 21);
    // joined sums of a row that both streams worked on: stream 1 hands its
    // part over through the ring
    float* part = reinterpret_cast<float*>(ring);  // [dim][row]
    float* s_m = part + D * kStreamRows;
    float* s_l = s_m + kStreamRows;
    float w0 = 1.f, w1 = 0.f;
    const bool two = !by_rows && tiles > 1;
    if (two) {
      if (st == 1) {
        s_m[rr] = m;
        s_l[rr] = l;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(to + c * 32, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) part[(c * 32 + i) * kStreamRows + rr] = __uint_as_float(v[i]);
        }
      }
      asm volatile("bar.sync 2, 256;" ::: "memory");
      if (st == 0) {
        const float m1 = s_m[rr], l1 = s_l[rr];
        const float top = fmaxf(m, m1), ref = top == neg_inf() ? 0.f : top;
        w0 = exp2f(m - ref);
        w1 = exp2f(m1 - ref);
        l = l * w0 + l1 * w1;
        m = top;
      }
    }
    const int row = by_rows ? st * kStreamRows + rr : rr;
    const bool mine = (by_rows || st == 0) && row < rows;
    if (by_rows || st == 0) {
      const int64_t t = rq.tok0 + token_of(mine ? row : 0);
      const int32_t head = head_of(mine ? row : 0);
      const bool none = l == 0.f || tiles == 0;
      const float inv = none ? 0.f : 1.f / l;
      const int64_t part_row = (int64_t(split) * a.num_tokens + t) * a.num_heads + head;
      const bool to_part = a.part_o != nullptr;
      uint16_t* out = a.out.data + t * a.out.ts + head * a.out.hs;
      const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;  // for 32-byte stores
      // A row is odd if keys past its limit were among its tiles and its sums
      // are not finite (0 * NaN), or if a block was bad.
      float check = l * 0.f;  // NaN once a sum is not finite
      const float scale = to_part ? w0 : w0 * inv, scale1 = to_part ? w1 : w1 * inv;
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) {
        float x[16];
        if (tiles > 0) {
          tmem_ld<16>(to + c * 16, *reinterpret_cast<uint32_t(*)[16]>(&x));
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = 0.f;
        }
        if (two) {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = fmaf(part[(c * 16 + i) * kStreamRows + rr], scale1, x[i] * scale);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] *= scale;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) check = fmaf(x[i], 0.f, check);
        if (!mine) continue;
        if (to_part) {
          float4* dst = reinterpret_cast<float4*>(a.part_o + part_row * D + c * 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        } else {
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = none ? 0u : to_bf16x2(x[2 * i], x[2 * i + 1]);
          if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + c * 16), "r"(o[0]),
                         "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                         : "memory");
          } else {
            st16(out + c * 16, make_uint4(o[0], o[1], o[2], o[3]));
            st16(out + c * 16 + 8, make_uint4(o[4], o[5], o[6], o[7]));
          }
        }
      }
      const bool odd = tiles > 0 && (s_bad != 0 || (lim < hi && check != 0.f));
      if (mine && to_part)
        a.part_ml[part_row] = make_float2(m, l);
      else if (mine && a.lse != nullptr)
        a.lse[t * a.num_heads + head] = none ? neg_inf() : (m + log2f(l)) * kLn2;
      // odd rows, one after the other by the whole warp, whose stores come
      // behind what the rows' own threads have stored above
      uint32_t todo = __ballot_sync(0xffffffffu, odd && mine);
      __syncwarp();
      while (todo) {
        const int from = __ffs(todo) - 1;
        todo &= todo - 1;
        const int64_t tt = __shfl_sync(0xffffffffu, t, from);
        const int32_t hh = __shfl_sync(0xffffffffu, head, from), top = __shfl_sync(0xffffffffu, lim, from);
        const int odd_row = __shfl_sync(0xffffffffu, row, from);
        float om, ol, o[D / 32];
        row_by_keys<D>(a, r, h, smem, odd_row, lo, top, om, ol, o);
        if (to_part) {
          const int64_t at = (int64_t(split) * a.num_tokens + tt) * a.num_heads + hh;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) a.part_o[at * D + lane + 32 * i] = o[i];
          if (lane == 0) a.part_ml[at] = make_float2(om, ol);
          continue;
        }
        const float scale = ol == 0.f ? 0.f : 1.f / ol;
        uint16_t* dst = a.out.data + tt * a.out.ts + hh * a.out.hs;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          dst[lane + 32 * i] = __bfloat16_as_ushort(__float2bfloat16_rn(ol == 0.f ? 0.f : o[i] * scale));
        if (lane == 0 && a.lse != nullptr)
          a.lse[tt * a.num_heads + hh] = ol == 0.f ? neg_inf() : (om + log2f(ol)) * kLn2;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == S::kProductWarp) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// The output of rows whose sums are in parts (of either attention kernel): one
// warp a row, the parts' weights a lane each.  Rows that no request owns, or a
// refused one, are left as they are.  It is a launch and two dependent loads:
// some 4 us behind the grid that writes the parts.
constexpr int kJoinRows = 8;  // of a CTA

template <int D>
__global__ void __launch_bounds__(kJoinRows * 32) join_parts_kernel(const __grid_constant__ AttendArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t part_rows = int64_t(a.num_tokens) * a.num_heads;
  const int64_t row = int64_t(blockIdx.x) * kJoinRows + threadIdx.x / 32;
  const int32_t t = int32_t(min(row, part_rows - 1) / a.num_heads), head = int32_t(row - int64_t(t) * a.num_heads);
  Request q;
  const bool owned =
      row < part_rows && read_request(a, owner_of(a, t), q) == 0 && t >= q.tok0 && t < q.tok0 + q.n;
  wait_for_previous();
  if (!owned) return;
  // lane k: part k's maximum and sum, then its weight
  float2 ml = make_float2(neg_inf(), 0.f);
  if (lane < a.num_parts) ml = __ldcg(&a.part_ml[lane * part_rows + row]);
  const float m = warp_max(ml.x);
  const float weight = exp2f(ml.x - (m == neg_inf() ? 0.f : m));
  float l = weight * ml.y, x[D / 32] = {};
#pragma unroll
  for (int d = 16; d > 0; d /= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
#pragma unroll 8
  for (int k = 0; k < a.num_parts; ++k) {
    const float w = __shfl_sync(0xffffffffu, weight, k);
    // nothing seen: the part's values mean nothing
    const bool seen = __shfl_sync(0xffffffffu, ml.y, k) != 0.f;
    const float* o = a.part_o + (k * part_rows + row) * D;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(o + 64 * i + 2 * lane));
      x[2 * i] = fmaf(w, seen ? v.x : 0.f, x[2 * i]);
      x[2 * i + 1] = fmaf(w, seen ? v.y : 0.f, x[2 * i + 1]);
    }
  }
  // a sum of 0: no key was seen, or none with a score above -inf
  const bool none = l == 0.f;
  const float inv = none ? 0.f : 1.f / l;
  uint16_t* out = a.out.data + t * a.out.ts + head * a.out.hs;
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
    *reinterpret_cast<uint32_t*>(out + 64 * i + 2 * lane) = none ? 0u : to_bf16x2(x[2 * i] * inv, x[2 * i + 1] * inv);
  if (a.lse != nullptr && lane == 0) a.lse[row] = none ? neg_inf() : (m + log2f(l)) * kLn2;
}

}  // namespace isq
