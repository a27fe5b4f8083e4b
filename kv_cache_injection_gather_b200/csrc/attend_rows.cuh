// Attention over the paged cache for few query rows per KV head (decode, a
// few speculated tokens): every key and value is read once and meets a few
// rows, so HBM bandwidth bounds it.
//
//   s_j = scale q . k_j,  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m)
//
// in one pass over the keys with a running reference m and sum, in base 2
// (scale * log2(e) is folded into one multiplier).  A unit of up to NR rows --
// the (token, head) pairs of one request that share a KV head -- meets tiles
// of 128 keys.  The keys take the 128-row side of the tensor cores and the
// rows the short one:
//
//   S^T = K Q^T   (128 keys x NR, in tensor memory)
//   P^T = exp2(scale S^T - m), to shared memory
//   O^T += V^T P  (D x NR or D x 2 NR, in tensor memory)
//
// The tensor cores take both operands in one type, so P is rounded to bf16: by
// itself an error of up to 2^-8 of sum p |v| beside the result's rounding.  For
// units of 16 rows the remainder of the rounding goes in as well, in columns of
// its own (V is read once for both) whose sums are added at the end.  Together
// they are within 2^-16 of P, and the result's rounding is the only one that
// counts; the tensor cores are 7% busy and decode takes 0-3% longer for it.
// Units of 32 rows (prompts with head_dim 32) would take a fifth longer (one of
// 2048 tokens 300 -> 353 us); they keep the rounded P.
//
// so that a tile costs the softmax threads, one key each, NR values and not a
// padded 128 (mma.sync over 16-row tiles spent 2900 cycles a warp and 32-key
// tile, an SM's whole share of the bandwidth).  Warps 0-3 do the softmax; the
// next bring keys and values, as TMA boxes of a block's tokens, into a ring
// of up to 192 KB; one thread of the last warp issues the products, the next
// tile's scores ahead of this tile's sums.  The keys of a unit can be split
// over a cluster, whose CTAs join their sums through distributed shared memory,
// and long ones over several clusters, whose sums a grid behind joins.
//
// Measured on B200 (32 query and 8 KV heads of 128, block 16): 100 requests of
// 800-3200 keys 143 us, 5.7 TB/s of keys and values, 0.89 of the copy
// bandwidth; 3 requests of 60-131 k keys (4 KV heads, 12 parts: 144 of 148 SMs)
// 117 us, 5.4 TB/s, as the longest one's parts end last.  A tile's rounded
// probabilities alone cost an SM some 1500 cycles, of 2200 that its share of the
// bandwidth leaves; a unit's start and end cost some 10 000, which is what bounds
// requests of a few hundred keys (100 of 550: 78 us, 2.9 TB/s).  With head_dim 32,
// 64 and 256 the 100 requests of 800-3200 keys take 109, 115 and 346 us (0.29,
// 0.55 and 0.74 of the copy bandwidth): a unit's start and end again, and at 256 a
// ring of three tiles.  Key by key (blocks of 5, 4, 1 tokens) they take 219, 228
// and 242 us, as a gather warp waits for each tile that it brings.
#pragma once

#include "attend_common.cuh"

namespace isq {

constexpr int kMostSplits = 8;   // CTAs of a cluster

template <int D, int NR>
struct RowsShape {
  static constexpr int kSlotBytes = kTileKeys * D * 2;         // one K or V tile
  // as many slots as fit, and gather warps that divide them
  static constexpr int kSlots = D == 256 ? 3 : D == 128 ? 6 : D == 64 ? 10 : 16;
  static constexpr int kGather = D == 32 ? 4 : D == 64 ? 5 : kSlots;
  static constexpr int kProductWarp = 4 + kGather;
  static constexpr int kThreads = (4 + kGather + 1) * 32;
  static constexpr int kQBytes = NR * D * 2;
  static constexpr bool kRest = NR == 16;
  static constexpr int kPRows = kRest ? 2 * NR : NR;           // rounded values, then remainders
  static constexpr int kPBytes = kPRows * kTileKeys * 2;       // twice
  static constexpr int kJoinBytes = NR * D * 4;                // the cluster's sums of this CTA's dims
  // Where shared memory has no room for both, the joined sums lie over P: other
  // CTAs may write them only once this one's products are done.
  static constexpr bool kJoinOverP = D == 256;
  static_assert(!kJoinOverP || kJoinBytes <= 2 * kPBytes, "the joined sums fit over P");
  static constexpr int kRingBytes = kSlots * kSlotBytes;
  static constexpr int kSmemBytes = kRingBytes + (kQBytes + 1023) / 1024 * 1024 + 2 * kPBytes +
                                    (kJoinOverP ? 0 : kJoinBytes) + 1024;
  static constexpr int kGroups = (D + 127) / 128;              // O^T accumulators, of kPRows columns
  // S^T twice and O^T, as a power of two of columns
  static constexpr int kColumns = 2 * NR + kGroups * kPRows <= 64 ? 64 : 128;
  static_assert(2 * NR + kGroups * kPRows <= kColumns, "tensor memory");
};

template <int D, int NR>
__global__ void __launch_bounds__(RowsShape<D, NR>::kThreads, 1) attend_rows_kernel(
    const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap k_map,
    const __grid_constant__ CUtensorMap v_map) {
  using S = RowsShape<D, NR>;
  constexpr int CPR = D / 8, NS = S::kSlots, NT = S::kThreads;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bar_full[NS], bar_empty[NS], bar_q, bar_s[2], bar_p[2], bar_o, bar_end;
  __shared__ __align__(16) float s_m[NR];
  __shared__ __align__(16) float s_top[4][NR], s_shrink[NR];
  __shared__ float s_l[NR];
  __shared__ __align__(8) float2 s_join_ml[kMostSplits][NR];  // of the cluster's CTAs
  __shared__ int32_t s_lim[NR], s_odd[NR];
  __shared__ uint32_t s_tmem;
  __shared__ int32_t s_failed, s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;

  // grid: x (KV head, part, split), the splits of a unit, head and part a
  // cluster; y and z the unit, of which the one after the last checks the batch
  if (a.key_parts > 1) let_next_start();
  const int32_t split = int32_t(blockIdx.x) & (a.splits - 1);
  const int32_t h = int32_t(blockIdx.x >> a.splits_log2) / a.key_parts;
  const int32_t part = int32_t(blockIdx.x >> a.splits_log2) - h * a.key_parts;
  const int64_t unit = int64_t(blockIdx.z) * gridDim.y + blockIdx.y;
  if (unit >= a.units) {
    if (unit == a.units && blockIdx.x == 0) check_requests<NT>(a);
    wait_for_previous();
    return;
  }
  // this CTA has started: its shared memory may be written
  if (!S::kJoinOverP && a.splits > 1) cluster_arrive();
  // what needs no metadata first, a barrier a thread
  if (tid < NS) {
    bar_init(&bar_full[tid], 1);
    bar_init(&bar_empty[tid], 1);
  } else if (tid >= 32 && tid < 34) {
    bar_init(&bar_s[tid - 32], 1);
    bar_init(&bar_p[tid - 32], 128);
  } else if (tid == 64) {
    bar_init(&bar_q, 128);
    bar_init(&bar_o, 1);
    bar_init(&bar_end, 1);
    s_failed = 0;
    s_bad = 0;
  } else if (tid == 96) {
    fetch_map(&k_map);
    fetch_map(&v_map);
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (warp == S::kProductWarp) tmem_alloc(&s_tmem, S::kColumns);
  int32_t r, tile;
  Request rq;
  find_unit<NR, NT>(a, int32_t(unit), r, tile, rq);
  if (r < 0) {  // so for the whole cluster
    if (warp == S::kProductWarp) tmem_free(s_tmem, S::kColumns);
    if (!S::kJoinOverP && a.splits > 1) cluster_wait();
    wait_for_previous();  // on every path: the next grid relies on both
    return;
  }

  const int32_t row0 = tile * NR;
  const int32_t rows = min(NR, rq.n * a.group - row0);
  auto token_of = [&](int row) { return (row0 + row) / a.group; };
  auto head_of = [&](int row) { return h * a.group + (row0 + row) % a.group; };
  // keys [lo, hi) of this CTA, of all [first_key, last row's limit): whole
  // tiles, from a box's border on (the keys below first_key are left out)
  const int32_t begin = a.box_log2 < 0 ? a.first_key : a.first_key >> a.box_log2 << a.box_log2;
  const int32_t end = row_limit(a, rq, token_of(rows - 1));
  const uint32_t all_tiles = end > a.first_key ? uint32_t(end - begin + kTileKeys - 1) / kTileKeys : 0;
  const uint32_t shares = a.key_parts << a.splits_log2, mine = (part << a.splits_log2) + split;
  // (below 2^24 tiles, times up to 2^8 shares)
  const int32_t lo = begin + int32_t(all_tiles * mine / shares) * kTileKeys;
  const uint32_t last = all_tiles * (mine + 1) / shares;
  const int32_t hi = all_tiles == 0 ? lo : last == all_tiles ? end : begin + int32_t(last) * kTileKeys;
  const int32_t tiles = hi > lo ? (hi - lo + kTileKeys - 1) / kTileKeys : 0;

  unsigned char* ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  unsigned char* p_tiles = ring + S::kRingBytes;
  float* join_o = reinterpret_cast<float*>(p_tiles + (S::kJoinOverP ? 0 : 2 * S::kPBytes));  // [split][row][D / splits]
  unsigned char* q_tile = p_tiles + 2 * S::kPBytes + (S::kJoinOverP ? 0 : S::kJoinBytes);

  if (tid < NR) {
    s_lim[tid] = tid < rows ? min(hi, row_limit(a, rq, token_of(tid))) : hi;
    // rows that are not there never rise above their reference
    s_m[tid] = tid < rows ? neg_inf() : -neg_inf();
    s_l[tid] = 0.f;
    s_shrink[tid] = 1.f;
    s_odd[tid] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;               // S^T, twice NR columns
  const uint32_t tmem_o = tmem + 2 * NR;      // O^T, kPRows columns per 128 dims

  if (warp >= 4 && warp < S::kProductWarp) {
    gather_tiles<D, NS, S::kGather>(a, &k_map, &v_map, warp - 4, r, h, lo, hi, tiles, ring, bar_full, bar_empty, nullptr,
                                    &s_failed, &s_bad);
  } else if (warp == S::kProductWarp) {
    // ---------------- products
    if (tiles > 0 && elect_one()) {
      bool ok = bar_wait(&bar_q, 0, &s_failed);
      auto wait_tile = [&](int32_t u) { ok = ok && bar_wait(&bar_full[u % NS], (u / NS) & 1, &s_failed); };
      auto scores = [&](int32_t t) {
        const int slot = (2 * t) % NS;
        wait_tile(2 * t);
        if (!ok) return;
        tc_fence_after();
        const uint32_t ka = smem_addr(ring + slot * S::kSlotBytes), qa = smem_addr(q_tile);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss(tmem + (t & 1) * NR, operand<D>(ka + dims_at<D>(k), 16), operand<D>(qa + dims_at<D>(k), 16),
                 product(NR, false, false), k > 0);
        tc_commit(&bar_s[t & 1]);
        tc_commit(&bar_empty[slot]);
      };
      scores(0);
      for (int32_t t = 0; t < tiles && ok; ++t) {
        if (t + 1 < tiles) scores(t + 1);
        ok = ok && bar_wait(&bar_p[t & 1], (t >> 1) & 1, &s_failed);
        const int slot = (2 * t + 1) % NS;
        wait_tile(2 * t + 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t va = smem_addr(ring + slot * S::kSlotBytes);
        const uint32_t pa = smem_addr(p_tiles + (t & 1) * S::kPBytes);
#pragma unroll
        for (int g = 0; g < S::kGroups; ++g)
#pragma unroll
          for (int k = 0; k < kTileKeys / 16; ++k)
            // V^T: 128 rows of dims; with D below 128 its slabs repeat (lead 0)
            mma_ss(tmem_o + g * S::kPRows, operand<D>(va + g * 2 * kSlabStep + k * (D * 32), D < 128 ? 0 : kSlabStep),
                   operand<128>(pa + dims_at<128>(k), 16), product(S::kPRows, true, false), t > 0 || k > 0);
        tc_commit(&bar_empty[slot]);
        tc_commit(&bar_o);
      }
      // All products are done before the threads meet: O is read then, and the
      // CTA may leave.  (bar_o cannot say so.  A parity tells phase n from n - 1
      // and n + 1, so a wait for n counts only where n - 1 is known to be done;
      // the last scores are issued ahead of the last but one sums, whose phase
      // nothing waits for.)
      tc_commit(&bar_end);
      if (!bar_wait(&bar_end, 0, nullptr)) s_failed = 1;
    }
    __syncwarp();
  } else {
    // ---------------- softmax, one key a thread
    load_queries<D>(q_tile, rows, NR, tid, 128, a.q.data, [&](int row) {
      return a.q.data + int64_t(rq.tok0 + token_of(row)) * a.q.ts + head_of(row) * a.q.hs;
    });
    bar_arrive(&bar_q);

    const int32_t lim_min = s_lim[0];  // limits rise with the rows
    const uint32_t lanes = uint32_t(warp) << 21;
    float l[NR];
#pragma unroll
    for (int c = 0; c < NR; ++c) l[c] = 0.f;
    // A warp whose wait gave up goes on without its tiles: the barriers below
    // are the four warps' together.
    bool ok = true;
    for (int32_t t = 0; t < tiles; ++t) {
      const int32_t j0 = lo + t * kTileKeys, j = j0 + tid;
      const bool edge = j0 < a.first_key || hi - j0 < kTileKeys;
      const bool in = j >= a.first_key && hi - j0 > tid;
      ok = ok && __all_sync(0xffffffffu, bar_wait(&bar_s[t & 1], (t >> 1) & 1, &s_failed));
      tc_fence_after();
      uint32_t v[NR];
      if (ok) {
        tmem_ld<NR>(tmem + (t & 1) * NR + lanes, v);
        tmem_wait_ld();
      }
      // Values of keys that take no part become zeros: their probabilities
      // are, and 0 * NaN is not.
      if (edge) {
        const int u = 2 * t + 1;
        ok = ok && __all_sync(0xffffffffu, bar_wait(&bar_full[u % NS], (u / NS) & 1, &s_failed));
        if (ok && !in) {
          unsigned char* row = ring + (u % NS) * S::kSlotBytes;
          for (int c = 0; c < CPR; ++c)
            *reinterpret_cast<uint4*>(row + tile_at<D>(tid, c)) = make_uint4(0, 0, 0, 0);
        }
      }
      const bool masked = edge || j0 + kTileKeys > lim_min;
      float x[NR];
      bool above = false;
      // The reference m of a row follows its maximum only when that has risen
      // by more than 2^8: smaller steps leave P below 2^8 and the sums as they
      // are.  (-inf + 8 is -inf: the first seen key counts.)
#pragma unroll
      for (int c = 0; c < NR; c += 4) {
        if (c >= rows) break;
        const float4 m4 = *reinterpret_cast<const float4*>(&s_m[c]);
        const float m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[c + i] = ok ? __uint_as_float(v[c + i]) * a.scale_log2 : neg_inf();
          if (masked && (!in || j >= s_lim[c + i])) x[c + i] = neg_inf();
          above = above || x[c + i] > m[i] + 8.f;
        }
      }
      uint32_t any;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\t"
          "selp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(any)
          : "r"(uint32_t(above))
          : "memory");
      if (any) {
#pragma unroll
        for (int c = 0; c < NR; c += 4) {
          if (c >= rows) break;
          float top[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) top[i] = warp_max(x[c + i]);
          if (lane == 0) *reinterpret_cast<float4*>(&s_top[warp][c]) = make_float4(top[0], top[1], top[2], top[3]);
        }
        asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
        if (tid < rows) {
          const float old = s_m[tid];
          const float top = fmaxf(fmaxf(fmaxf(s_top[0][tid], s_top[1][tid]), fmaxf(s_top[2][tid], s_top[3][tid])), old);
          s_m[tid] = top;
          s_shrink[tid] = top == neg_inf() ? 1.f : exp2_fast(old - top);
        }
        asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
        // (the sums up to t - 2 are done, as a wait for phase t - 1 needs: their
        // commit came before that of this tile's scores)
        if (t > 0) ok = ok && __all_sync(0xffffffffu, bar_wait(&bar_o, (t - 1) & 1, &s_failed));
        if (t > 0 && ok) {
          tc_fence_after();
          float shrink[NR];
#pragma unroll
          for (int c = 0; c < NR; c += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&s_shrink[c]);
            shrink[c] = f.x, shrink[c + 1] = f.y, shrink[c + 2] = f.z, shrink[c + 3] = f.w;
          }
#pragma unroll
          for (int c = 0; c < NR; ++c) l[c] *= shrink[c];
#pragma unroll
          for (int g = 0; g < S::kGroups * S::kPRows / NR; ++g) {
            tmem_ld<NR>(tmem_o + g * NR + lanes, v);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < NR; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * shrink[c]);
            tmem_st<NR>(tmem_o + g * NR + lanes, v);
          }
          tmem_wait_st();
        }
      }
      // P^T as the second product's B operand: a tile of [row][128 keys], the
      // rows' values rounded to bf16 and, NR rows on, what that left out (kRest;
      // the difference is exact).
      unsigned char* p = p_tiles + (t & 1) * S::kPBytes + (tid & 7) * 2;
#pragma unroll
      for (int c = 0; c < NR; c += 4) {
        if (c >= rows) break;  // the products of other rows are not looked at
        const float4 m4 = *reinterpret_cast<const float4*>(&s_m[c]);
        const float m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = exp2_fast(x[c + i] - (m[i] == neg_inf() ? 0.f : m[i]));  // no key seen yet: every term is 0
          l[c + i] += e;
          const __nv_bfloat16 near = __float2bfloat16_rn(e);
          *reinterpret_cast<uint16_t*>(p + tile_at<128>(c + i, tid >> 3)) = __bfloat16_as_ushort(near);
          if constexpr (S::kRest)
            *reinterpret_cast<uint16_t*>(p + tile_at<128>(NR + c + i, tid >> 3)) =
                __bfloat16_as_ushort(__float2bfloat16_rn(e - __bfloat162float(near)));
        }
      }
      proxy_fence();
      tc_fence_before();
      bar_arrive(&bar_p[t & 1]);
    }
    // ---- the CTA's sums
#pragma unroll
    for (int c = 0; c < NR; c += 4) {
      if (c >= rows) break;
#pragma unroll
      for (int d = 16; d > 0; d /= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) l[c + i] += __shfl_xor_sync(0xffffffffu, l[c + i], d);
      if (lane == 0) *reinterpret_cast<float4*>(&s_top[warp][c]) = make_float4(l[c], l[c + 1], l[c + 2], l[c + 3]);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // a row is odd if its sums are not finite and keys past its limit were in
  // its tiles, or if a block was bad: it is summed again key by key
  uint32_t o[S::kGroups][NR];
  if (warp < 4) {
    if (tid < rows) s_l[tid] = s_top[0][tid] + s_top[1][tid] + s_top[2][tid] + s_top[3][tid];
#pragma unroll
    for (int g = 0; g < S::kGroups; ++g) {
      if (tiles > 0) {
        tmem_ld<NR>(tmem_o + g * S::kPRows + (uint32_t(warp) << 21), o[g]);
        if constexpr (S::kRest) {
          uint32_t rest[NR];
          tmem_ld<NR>(tmem_o + g * S::kPRows + NR + (uint32_t(warp) << 21), rest);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < NR; ++c)
            o[g][c] = __float_as_uint(__uint_as_float(o[g][c]) + __uint_as_float(rest[c]));
        }
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int c = 0; c < NR; ++c) o[g][c] = 0;
      }
#pragma unroll
      for (int c = 0; c < NR; ++c)
        if (c < rows && g * 128 + tid < D && !finite(__uint_as_float(o[g][c])) && s_lim[c] < hi) s_odd[c] = 1;
    }
    if (s_bad != 0 && tid < rows) s_odd[tid] = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == S::kProductWarp) {
    tc_fence_after();
    tmem_free(tmem, S::kColumns);
  }

  // ---- join the splits: CTA k of the cluster gets everybody's maxima and sums
  // and the k-th share of the dims, written into its shared memory
  if (S::kJoinOverP && a.splits > 1) cluster_arrive();  // this CTA's products are done
  if (a.splits > 1) cluster_wait();  // so are all CTAs', or they have all started
  constexpr int kLogD = D == 256 ? 8 : D == 128 ? 7 : D == 64 ? 6 : 5;
  const int share_log2 = kLogD - a.splits_log2, share = 1 << share_log2;
  const uint32_t o_at = smem_addr(join_o), ml_at = smem_addr(s_join_ml);
  // of (row 0, dim d) in the CTA that gets it; rows are 4 * share bytes apart
  auto join_at = [&](int d) {
    return in_cta(o_at + (((split * NR << share_log2) + (d & (share - 1))) << 2), d >> share_log2);
  };
  auto join_ml = [&](int row, float m, float l, int to) {
    st_cluster2(in_cta(ml_at + (split * NR + row) * 8, to), m, l);
  };
  if (warp < 4) {
#pragma unroll
    for (int g = 0; g < S::kGroups; ++g) {
      if (g * 128 + tid >= D) break;
      const uint32_t to = join_at(g * 128 + tid);
#pragma unroll
      for (int c = 0; c < NR; ++c) {
        if (c >= rows) break;
        if (!s_odd[c]) st_cluster(to + (c << (share_log2 + 2)), __uint_as_float(o[g][c]));
      }
    }
  } else {
    for (int i = tid - 128; i < rows << a.splits_log2; i += NT - 128) {
      const int row = i >> a.splits_log2;
      if (!s_odd[row]) join_ml(row, s_m[row], s_l[row], i & (a.splits - 1));
    }
  }
  for (int row = warp; row < rows; row += NT / 32) {
    if (!s_odd[row]) continue;
    float m, l, x[D / 32];
    row_by_keys<D>(a, r, h, q_tile, row, max(lo, a.first_key), s_lim[row], m, l, x);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) st_cluster(join_at(lane + 32 * i) + (row << (share_log2 + 2)), x[i]);
    if (lane < a.splits) join_ml(row, m, l, lane);
  }
  if (a.splits > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  wait_for_previous();
  const int64_t part_rows = int64_t(a.num_tokens) * a.num_heads;
  for (int i = tid; i < rows << (share_log2 - 2); i += NT) {
    const int row = i >> (share_log2 - 2), c = (i << 2) & (share - 1);
    const int64_t t = rq.tok0 + token_of(row);
    const int32_t head = head_of(row), d = split * share + c;
    const int64_t part_row = t * a.num_heads + head;
    float m = neg_inf();
    for (int k = 0; k < a.splits; ++k) m = fmaxf(m, s_join_ml[k][row].x);
    for (int k = 0; k < a.num_parts; ++k) m = fmaxf(m, __ldcg(&a.part_ml[k * part_rows + part_row].x));
    const float ref = m == neg_inf() ? 0.f : m;
    float l = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < a.splits; ++k) {
      const float2 ml = s_join_ml[k][row];
      const float w = exp2f(ml.x - ref);
      const float4 v = *reinterpret_cast<const float4*>(join_o + ((k * NR + row) << share_log2) + c);
      l += w * ml.y;
      sum.x = fmaf(w, v.x, sum.x);
      sum.y = fmaf(w, v.y, sum.y);
      sum.z = fmaf(w, v.z, sum.z);
      sum.w = fmaf(w, v.w, sum.w);
    }
    for (int k = 0; k < a.num_parts; ++k) {
      const float2 ml = __ldcg(&a.part_ml[k * part_rows + part_row]);
      const float w = exp2f(ml.x - ref);
      if (ml.y == 0.f) continue;  // nothing seen: the part's values mean nothing
      l += w * ml.y;
      const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + (k * part_rows + part_row) * D + d));
      sum.x = fmaf(w, v.x, sum.x);
      sum.y = fmaf(w, v.y, sum.y);
      sum.z = fmaf(w, v.z, sum.z);
      sum.w = fmaf(w, v.w, sum.w);
    }
    if (a.key_parts > 1) {
      const int64_t at = part * part_rows + part_row;
      *reinterpret_cast<float4*>(a.part_o + at * D + d) = sum;
      if (d == 0) a.part_ml[at] = make_float2(m, l);
      continue;
    }
    // a sum of 0: no key was seen, or none with a score above -inf
    const bool none = l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
    if (none) sum = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<uint2*>(a.out.data + t * a.out.ts + head * a.out.hs + d) =
        make_uint2(to_bf16x2(sum.x * inv, sum.y * inv), to_bf16x2(sum.z * inv, sum.w * inv));
    if (a.lse != nullptr && d == 0) a.lse[part_row] = none ? neg_inf() : (m + log2f(l)) * kLn2;
  }
  if (s_failed && tid == 0) record(a.st, kErrTimeout, r);
}

}  // namespace isq
