// Attention over the paged cache for few query rows per KV head (decode, a
// few speculated tokens): the keys and values are read once and stream past
// the rows, so HBM bandwidth bounds it.
//
//   s_j = scale q . k_j,  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m)
//
// in one pass over the keys with the running maximum m and sum, in base 2
// (scale * log2(e) is folded into one multiplier).  A tile of up to 16 rows
// -- the (token, head) pairs of one request that share a KV head -- is the M
// side of mma.m16n8k16 (bf16 in, fp32 out).  Each warp of a CTA walks its own
// keys with its own ring of tiles, m, sum and accumulator, so the loop has no
// CTA-wide barrier; the warps' parts are joined at the end.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "query_rows.cuh"

namespace isq {

struct AttendArgs {
  int32_t num_tokens, num_requests, max_q_len, max_blocks;
  const int32_t* q_offsets;
  const int32_t* start_pos;
  const int32_t* kv_lens;
  const int32_t* block_tables;
  const int32_t* shared_blocks;
  int32_t shared_len;
  int32_t causal;
  int32_t splits;              // CTAs that share a unit's keys
  // Parts of the rows' sums in the work space, each [num_tokens][num_heads]:
  // (maximum, sum) pairs and [D] sums of values, all fp32.  attend_tiles
  // writes part `split`; attend_rows reads `num_parts` of them.
  float2* part_ml;
  float* part_o;
  int32_t num_parts;
  int32_t first_key;           // attend_rows: the keys below are in the parts
  int32_t table_shared;        // positions below are looked up in shared_blocks
  // Keys of one tensor-map box (a power of two that divides the block size and
  // the kernel's tile), as a logarithm; -1: gather by rows.
  int32_t box_log2;
  float scale_log2;            // scale * log2(e)
  int32_t num_heads;           // query heads
  int32_t group;               // query heads per KV head
  int32_t kv_heads;
  Rows q, out;
  float* lse;
  // paged cache, at the layer
  const uint16_t* k_cache;
  const uint16_t* v_cache;
  int64_t block_stride, token_stride, head_stride;
  int32_t num_blocks, block_size;
  Status* st;
};

constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __uint_as_float(0x7f800000u); }

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16 bytes global -> shared; `bytes` 16, or 0 to write zeros and read nothing.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- barriers

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// Waits until the phase of the given parity has completed.  After the limit
// (about two seconds), or once another thread has given up, returns false;
// without a flag only the limit counts.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int32_t* failed) {
  const uint32_t addr = smem_addr(bar);
  const long long began = clock64();
  while (true) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    if (done) return true;
    if (failed != nullptr && *failed) return false;
    if (clock64() - began > (1ll << 32)) {
      if (failed != nullptr) *failed = 1;
      return false;
    }
  }
}

// One arrival that also announces bytes.
__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
// One arrival, when this thread's cp.async so far have landed.
__device__ __forceinline__ void bar_arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// A box of the paged cache to shared memory: dims from `x`, tokens from `token`
// of block `block`, KV head h.  x is a multiple of 64 (or 0).
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t token, int32_t block,
                                         int32_t h, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(dst),
      "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(token), "r"(block), "r"(h)
      : "memory");
}
__device__ __forceinline__ void fetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Orders this thread's plain accesses to shared memory before later
// asynchronous ones (copies, tensor-core operands).
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- launches

// Programmatic dependent launch: the next grid on the stream may start; wait
// until the grid before is done (at once where there is none).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared variable in another CTA of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// ---------------------------------------------------------------- requests

struct Request {
  int32_t tok0, n;      // its query tokens
  int32_t start, kv;    // position of the first, keys in the cache
};

// Reads request r; 0, or the error that makes the batch skip it.
__device__ __forceinline__ int32_t read_request(const AttendArgs& a, int32_t r, Request& q) {
  const int32_t t0 = a.q_offsets[r], t1 = a.q_offsets[r + 1];
  q.start = a.start_pos[r];
  q.kv = a.kv_lens[r];
  q.tok0 = t0;
  q.n = t1 - t0;
  if (t0 < 0 || t1 < t0 || t1 > a.num_tokens || q.n > a.max_q_len || q.start < 0 || q.kv < 0)
    return kErrInvalidArg;
  if (q.kv > a.shared_len && q.kv > int64_t(a.max_blocks) * a.block_size) return kErrPosition;
  return 0;
}

// Position of query i of a request that is the first it does not see.
__device__ __forceinline__ int32_t row_limit(const AttendArgs& a, const Request& q, int32_t i) {
  if (!a.causal) return q.kv;
  const int64_t lim = int64_t(q.start) + i + 1;
  return lim < q.kv ? int32_t(lim) : q.kv;
}

// The request and row tile of work unit `unit`: the units are the requests'
// tiles of ROWS rows (row = token * group + head), in order.  The whole CTA
// calls this; r is -1 where there is no such unit.  Requests that read_request
// refuses have no unit.
template <int ROWS, int NT>
__device__ __forceinline__ void find_unit(const AttendArgs& a, int32_t unit, int32_t& r, int32_t& tile, Request& q) {
  if (int64_t(a.max_q_len) * a.group <= ROWS) {  // one tile each: the unit is the request
    r = -1;
    tile = 0;
    if (unit < a.num_requests && read_request(a, unit, q) == 0 && q.n > 0) r = unit;
    return;
  }
  __shared__ int32_t s_warp[NT / 32];
  __shared__ int32_t s_found[6];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  if (tid == 0) s_found[0] = -1;
  int32_t base = 0;
  for (int32_t r0 = 0; r0 < a.num_requests; r0 += NT) {
    Request mine;
    int32_t tiles = 0;
    if (r0 + tid < a.num_requests && read_request(a, r0 + tid, mine) == 0)
      tiles = int32_t((int64_t(mine.n) * a.group + ROWS - 1) / ROWS);
    int32_t upto = tiles;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int32_t o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    __syncthreads();  // s_warp of the round before is read
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    int32_t before = base, total = base;
    for (int i = 0; i < NT / 32; ++i) {
      if (i < warp) before += s_warp[i];
      total += s_warp[i];
    }
    upto += before;
    if (unit >= upto - tiles && unit < upto) {
      s_found[0] = r0 + tid;
      s_found[1] = unit - (upto - tiles);
      s_found[2] = mine.tok0;
      s_found[3] = mine.n;
      s_found[4] = mine.start;
      s_found[5] = mine.kv;
    }
    base = total;
    if (unit < total) break;
  }
  __syncthreads();
  r = s_found[0];
  tile = s_found[1];
  q.tok0 = s_found[2];
  q.n = s_found[3];
  q.start = s_found[4];
  q.kv = s_found[5];
}

// Records the first refused request of the batch; one CTA of a grid does it.
template <int NT>
__device__ __forceinline__ void check_requests(const AttendArgs& a) {
  __shared__ int32_t s_first;
  if (threadIdx.x == 0) s_first = INT32_MAX;
  __syncthreads();
  Request q;
  for (int32_t r = threadIdx.x; r < a.num_requests; r += NT)
    if (read_request(a, r, q) != 0) {
      atomicMin(&s_first, r);
      break;
    }
  __syncthreads();
  if (threadIdx.x == 0 && s_first != INT32_MAX) record(a.st, read_request(a, s_first, q), s_first);
}

// Table entry of position j (below the request's limit): the shared list's
// below table_shared, the request's own otherwise.
__device__ __forceinline__ int32_t table_entry(const AttendArgs& a, int32_t r, int32_t j) {
  const int32_t jb = j / a.block_size;
  return j < a.table_shared ? a.shared_blocks[jb] : a.block_tables[int64_t(r) * a.max_blocks + jb];
}
// Element offset of (position j in block `entry`, KV head h) in the layer's
// caches; -1 for a block outside the cache, which is recorded.
__device__ __forceinline__ int64_t entry_offset(const AttendArgs& a, int32_t r, int32_t h, int32_t j, int32_t entry) {
  if (entry < 0 || entry >= a.num_blocks) {
    record(a.st, kErrBadBlock, j < a.table_shared ? -1 : r);
    return -1;
  }
  return entry * a.block_stride + int64_t(j % a.block_size) * a.token_stride + h * a.head_stride;
}
__device__ __forceinline__ int64_t key_offset(const AttendArgs& a, int32_t r, int32_t h, int32_t j) {
  return entry_offset(a, r, h, j, table_entry(a, r, j));
}

// One row over keys [lo, hi) by a warp, key after key in fp32: for rows whose
// tiled product came out infinite or NaN although keys that they do not see
// may have caused it (0 * NaN).  o: dims lane, lane + 32, ...
template <int D>
__device__ __noinline__ void row_by_keys(const AttendArgs& a, int32_t r, int32_t h, const uint16_t* q, int32_t lo,
                                         int32_t hi, float& m, float& l, float (&o)[D / 32]) {
  const int lane = threadIdx.x & 31;
  float x[D / 32];
  m = neg_inf();
  l = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    x[i] = __uint_as_float(uint32_t(q[lane + 32 * i]) << 16);
    o[i] = 0.f;
  }
  for (int32_t j = lo; j < hi; ++j) {
    const int64_t at = key_offset(a, r, h, j);
    if (at < 0) continue;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      s = fmaf(x[i], __uint_as_float(uint32_t(a.k_cache[at + lane + 32 * i]) << 16), s);
#pragma unroll
    for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale_log2;
    const float top = fmaxf(m, s);
    const float ref = top == neg_inf() ? 0.f : top;
    const float shrink = exp2f(m - ref), p = exp2f(s - ref);
    m = top;
    l = l * shrink + p;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      o[i] = o[i] * shrink + p * __uint_as_float(uint32_t(a.v_cache[at + lane + 32 * i]) << 16);
  }
}

// ---------------------------------------------------------------- the kernel

constexpr int kTileRows = 16;

#ifndef V_KEYS
#define V_KEYS 32
#endif
#ifndef V_WARPS
#define V_WARPS 4
#endif
#ifndef V_STAGES
#define V_STAGES 3
#endif
template <int D>
struct RowsShape {
  static constexpr int kKeys = D <= 128 ? V_KEYS : 16;       // keys of a warp's tile
  static constexpr int kWarps = V_WARPS;
  static constexpr int kStages = V_STAGES;
  // A tile is D / 64 slabs of [keys][64 dims] (one of 32 dims for D = 32), as
  // a tensor-map box with its row as the swizzle's width leaves them.
  static constexpr int kSlabDims = D < 64 ? D : 64;
  static constexpr int kSlabs = D / kSlabDims;
  static constexpr int kSlabBytes = kKeys * kSlabDims * 2;
  static constexpr int kTileBytes = kSlabs * kSlabBytes;  // K or V
  static constexpr int kWarpBytes = kStages * 2 * kTileBytes;
  static constexpr int kRingBytes = kWarps * kWarpBytes;
  static constexpr int kQBytes = kTileRows * D * 2;
  static constexpr int kSmemBytes = kRingBytes + kQBytes + 1024;  // data, and up to 1 KB to align it
};

// Byte offset of 16-byte chunk c of row `row` in a tile of `keys` rows: the
// chunks of a slab's row are permuted by the row's number (the 128-byte
// swizzle; the 64-byte one for D = 32), so that 8 consecutive rows at one
// chunk, an ldmatrix phase, fall into different banks.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int keys, int row, int c) {
  if constexpr (D < 64) return uint32_t(row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
  return uint32_t((c >> 3) * keys * 128 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

template <int D>
__global__ void __launch_bounds__(RowsShape<D>::kWarps * 32) attend_rows_kernel(
    const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap k_map,
    const __grid_constant__ CUtensorMap v_map) {
  using S = RowsShape<D>;
  constexpr int NT = S::kWarps * 32, TK = S::kKeys, CPR = D / 8, KS = D / 16, NK = TK / 8, ND = D / 8;
  constexpr int SL = S::kSlabs;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  unsigned char* ring = smem + warp * S::kWarpBytes;
  unsigned char* q_tile = smem + S::kRingBytes;
  __shared__ float s_m[S::kWarps][kTileRows], s_l[S::kWarps][kTileRows];
  __shared__ float s_cta_m[kTileRows], s_cta_l[kTileRows];
  __shared__ int32_t s_odd[kTileRows];
  __shared__ __align__(8) uint64_t s_bar[S::kWarps][S::kStages];
  __shared__ int32_t s_failed;

  // grid: (unit, KV head, split), the splits of a unit and head a cluster; the
  // cluster after the last checks the batch
  const int32_t split = int32_t(blockIdx.x % a.splits);
  const int32_t cluster = int32_t(blockIdx.x / a.splits);
  const int32_t h = cluster % a.kv_heads;
  if (cluster == gridDim.x / a.splits - 1) {
    if (split == 0) check_requests<NT>(a);
    wait_for_previous();
    return;
  }
  int32_t r, tile;
  Request rq;
  find_unit<kTileRows, NT>(a, cluster / a.kv_heads, r, tile, rq);
  if (r < 0) {  // so for the whole cluster
    wait_for_previous();  // on every path: the next grid relies on both
    return;
  }

  const int32_t row0 = tile * kTileRows;
  const int32_t rows = min(kTileRows, rq.n * a.group - row0);
  auto token_of = [&](int row) { return (row0 + row) / a.group; };
  auto head_of = [&](int row) { return h * a.group + (row0 + row) % a.group; };
  // keys [lo, hi) of this CTA, of all [first_key, last row's limit): whole
  // tiles, from a box's border on (the keys below first_key are left out)
  const int32_t begin = a.box_log2 < 0 ? a.first_key : a.first_key >> a.box_log2 << a.box_log2;
  const int32_t end = row_limit(a, rq, token_of(rows - 1));
  const int64_t all_tiles = end > a.first_key ? (int64_t(end) - begin + TK - 1) / TK : 0;
  const int32_t lo = begin + int32_t(all_tiles * split / a.splits) * TK;
  const int32_t hi = int32_t(min(int64_t(end), begin + all_tiles * (split + 1) / a.splits * TK));

  // ---- the queries, as the A operand of every product
  for (int i = tid; i < kTileRows * CPR; i += NT) {
    const int row = i / CPR, c = i % CPR;
    const bool live = row < rows;
    const uint16_t* src = a.q.data;
    if (live) src += int64_t(rq.tok0 + token_of(row)) * a.q.ts + head_of(row) * a.q.hs + c * 8;
    cp_async16(smem_addr(q_tile + tile_at<D>(kTileRows, row, c)), src, live ? 16 : 0);
  }

  // ---- key tiles of this warp: tile i covers [lo + i * TK, ...), i = warp,
  // warp + kWarps, ...
  const int32_t tiles = hi > lo ? (hi - lo + TK - 1) / TK : 0;
  // A tile comes as boxes (op = lane: box lane / (2 SL), then K or V, then the
  // slab), or key by key where it holds keys of two blocks in one box.
  constexpr uint32_t kAll = TK == 32 ? 0xffffffffu : (1u << TK) - 1u;
  const int32_t my_box = lane / (2 * SL) << max(0, a.box_log2);  // first key of this lane's box
  auto by_box = [&](int32_t j0) {
    const bool torn = j0 < a.table_shared && a.table_shared - j0 < TK &&
                      (a.table_shared & ((1 << max(0, a.box_log2)) - 1)) != 0;
    return a.box_log2 >= 0 && !torn;
  };
  // The position that a lane looks up for tile i (-1: none) and its table
  // entry, read one tile ahead of the copies that need it.
  auto position = [&](int32_t i) -> int32_t {
    if (i >= tiles) return -1;
    const int32_t j0 = lo + i * TK, at = by_box(j0) ? my_box : lane;
    return at < TK && hi - j0 > at ? j0 + at : -1;
  };
  int32_t next_pos = position(warp);
  int32_t next_entry = next_pos < 0 ? 0 : table_entry(a, r, next_pos);

  // Starts the copies of tile i into a stage; returns which of its keys take
  // part.
  auto load = [&](int32_t i, int stage) -> uint32_t {
    const int32_t pos = next_pos, entry = next_entry;
    next_pos = position(i + S::kWarps);
    if (next_pos >= 0) next_entry = table_entry(a, r, next_pos);
    if (i >= tiles) return 0;
    const int32_t j0 = lo + i * TK;
    uint64_t* bar = &s_bar[warp][stage];
    const uint32_t k_dst = smem_addr(ring + stage * 2 * S::kTileBytes);
    bool good = pos >= 0 && entry >= 0 && entry < a.num_blocks;
    if (pos >= 0 && !good) record(a.st, kErrBadBlock, pos < a.table_shared ? -1 : r);
    if (by_box(j0)) {
      const uint32_t ops = __ballot_sync(0xffffffffu, good);
      if (lane == 0) bar_expect(bar, (uint32_t(__popc(ops)) << a.box_log2) * (S::kSlabDims * 2));
      else bar_arrive(bar);
      if (good) {
        const int slab = lane % SL;
        const bool v = (lane / SL) & 1;
        copy_box(k_dst + (v ? S::kTileBytes : 0) + slab * S::kSlabBytes + my_box * (S::kSlabDims * 2),
                 v ? &v_map : &k_map, slab * S::kSlabDims, pos % a.block_size, entry, h, bar);
      }
      const int32_t j = j0 + lane;
      const bool in = lane < TK && lane < hi - j0 && j >= a.first_key &&
                      ((ops >> ((lane >> a.box_log2) * (2 * SL) & 31)) & 1u);
      return __ballot_sync(0xffffffffu, in);
    }
    good = good && pos >= a.first_key;
    const int64_t at = good ? entry * a.block_stride + int64_t(pos % a.block_size) * a.token_stride + h * a.head_stride
                            : -1;
    const uint32_t ok = __ballot_sync(0xffffffffu, good);
#pragma unroll 4
    for (int n = 0; n < TK * CPR / 32; ++n) {
      const int e = n * 32 + lane, row = e / CPR, c = e % CPR;
      const int64_t from = __shfl_sync(0xffffffffu, at, row);
      const int64_t src = from < 0 ? 0 : from + c * 8;
      const int bytes = from < 0 ? 0 : 16;
      const uint32_t dst = k_dst + tile_at<D>(TK, row, c);
      cp_async16(dst, a.k_cache + src, bytes);
      cp_async16(dst + S::kTileBytes, a.v_cache + src, bytes);
    }
    bar_arrive_after_copies(bar);
    return ok;
  };

  if (lane == 0) {
    for (int s = 0; s < S::kStages; ++s) bar_init(&s_bar[warp][s], 32);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 0) {
    s_failed = 0;
    fetch_map(&k_map);
    fetch_map(&v_map);
  }
  __syncwarp();
  // which keys of the tiles in flight take part, the current tile's first
  uint32_t seen[S::kStages];
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) seen[s] = load(warp + s * S::kWarps, s);
  cp_async_commit();
  cp_async_wait<0>();  // the queries
  __syncthreads();
  uint32_t qf[KS][4];
#pragma unroll
  for (int k = 0; k < KS; ++k)
    ldmatrix4(qf[k], smem_addr(q_tile + tile_at<D>(kTileRows, lane & 15, 2 * k + (lane >> 4))));

  // rows lane / 4 and lane / 4 + 8 of the accumulators
  const int ra = lane >> 2, rb = ra + 8;
  const int32_t lim_a = ra < rows ? row_limit(a, rq, token_of(ra)) : hi;
  const int32_t lim_b = rb < rows ? row_limit(a, rq, token_of(rb)) : hi;
  const int32_t lim_min = row_limit(a, rq, token_of(0));
  float m_a = neg_inf(), m_b = neg_inf(), l_a = 0.f, l_b = 0.f;
  float o[ND][4];
#pragma unroll
  for (int i = 0; i < ND; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

  int stage = 0;
  uint32_t parity = 0;
  int32_t i = warp;
  for (; i < tiles; i += S::kWarps) {
    const int free_stage = stage == 0 ? S::kStages - 1 : stage - 1;  // the one read last
    __syncwarp();
    seen[S::kStages - 1] = load(i + (S::kStages - 1) * S::kWarps, free_stage);
    const uint32_t ok = seen[0];
#pragma unroll
    for (int s = 0; s < S::kStages - 1; ++s) seen[s] = seen[s + 1];
    if (!__all_sync(0xffffffffu, bar_wait(&s_bar[warp][stage], parity, &s_failed))) break;
    const unsigned char* kt = ring + stage * 2 * S::kTileBytes;
    const unsigned char* vt = kt + S::kTileBytes;
    // The values of keys that take no part become zeros: their probabilities
    // are, and 0 * NaN is not.
    if (ok != kAll) {
      if (lane < TK && !((ok >> lane) & 1u)) {
        unsigned char* row = ring + stage * 2 * S::kTileBytes + S::kTileBytes;
        for (int c = 0; c < CPR; ++c) *reinterpret_cast<uint4*>(row + tile_at<D>(TK, lane, c)) = make_uint4(0, 0, 0, 0);
        proxy_fence();  // before later copies to the stage
      }
      __syncwarp();
    }

    float s[NK][4];
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int n = 0; n < NK; n += 2) {
        uint32_t b[4];  // keys 8n .. 8n + 15, dims 16k .. 16k + 15
        ldmatrix4(b, smem_addr(kt + tile_at<D>(TK, n * 8 + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1))));
        mma16816(s[n], qf[k], b[0], b[1]);
        mma16816(s[n + 1], qf[k], b[2], b[3]);
      }

    const int32_t j0 = lo + i * TK;
    if (ok != kAll || j0 + TK > lim_min) {
#pragma unroll
      for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = n * 8 + (lane & 3) * 2 + (e & 1);
          if (!((ok >> col) & 1u) || j0 + col >= (e < 2 ? lim_a : lim_b)) s[n][e] = neg_inf();
        }
    }
    float top_a = s[0][0], top_b = s[0][2];
#pragma unroll
    for (int n = 0; n < NK; ++n) {
      top_a = fmaxf(top_a, fmaxf(s[n][0], s[n][1]));
      top_b = fmaxf(top_b, fmaxf(s[n][2], s[n][3]));
    }
    top_a *= a.scale_log2;  // positive: the maximum's place is the same
    top_b *= a.scale_log2;
    // The reference m follows the maximum only when that has risen by more
    // than 2^8: smaller steps leave p below 2^8 and the sums as they are.
    if (__any_sync(0xffffffffu, top_a > m_a + 8.f || top_b > m_b + 8.f)) {
#pragma unroll
      for (int d = 1; d < 4; d *= 2) {
        top_a = fmaxf(top_a, __shfl_xor_sync(0xffffffffu, top_a, d));
        top_b = fmaxf(top_b, __shfl_xor_sync(0xffffffffu, top_b, d));
      }
      top_a = fmaxf(top_a, m_a);
      top_b = fmaxf(top_b, m_b);
      const float shrink_a = top_a == neg_inf() ? 1.f : exp2_fast(m_a - top_a);
      const float shrink_b = top_b == neg_inf() ? 1.f : exp2_fast(m_b - top_b);
      m_a = top_a;
      m_b = top_b;
      l_a *= shrink_a;
      l_b *= shrink_b;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        o[d][0] *= shrink_a;
        o[d][1] *= shrink_a;
        o[d][2] *= shrink_b;
        o[d][3] *= shrink_b;
      }
    }
    // a row that has seen nothing yet: subtract 0, every term is 0
    const float ref_a = m_a == neg_inf() ? 0.f : m_a, ref_b = m_b == neg_inf() ? 0.f : m_b;
#pragma unroll
    for (int n = 0; n < NK; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = exp2_fast(fmaf(s[n][e], a.scale_log2, e < 2 ? -ref_a : -ref_b));
      l_a += s[n][0] + s[n][1];
      l_b += s[n][2] + s[n][3];
    }
#pragma unroll
    for (int k = 0; k < TK / 16; ++k) {
      // the probabilities rounded to bf16: the products' other operand, V, is
      // no finer, and the sum l keeps them in fp32
      const uint32_t p[4] = {to_bf16x2(s[2 * k][0], s[2 * k][1]), to_bf16x2(s[2 * k][2], s[2 * k][3]),
                             to_bf16x2(s[2 * k + 1][0], s[2 * k + 1][1]), to_bf16x2(s[2 * k + 1][2], s[2 * k + 1][3])};
#pragma unroll
      for (int d = 0; d < ND; d += 2) {
        uint32_t b[4];  // keys 16k .. 16k + 15, dims 8d .. 8d + 15
        ldmatrix4_trans(b, smem_addr(vt + tile_at<D>(TK, k * 16 + (lane & 15), d + (lane >> 4))));
        mma16816(o[d], p, b[0], b[1]);
        mma16816(o[d + 1], p, b[2], b[3]);
      }
    }
    if (++stage == S::kStages) {
      stage = 0;
      parity ^= 1;
    }
  }

  // after a wait that gave up: this warp's copies in flight
  for (int n = 0; n < S::kStages && i < tiles; ++n, i += S::kWarps) {
    bar_wait(&s_bar[warp][stage], parity, nullptr);
    if (++stage == S::kStages) {
      stage = 0;
      parity ^= 1;
    }
  }

  // ---- join the warps' parts
#pragma unroll
  for (int d = 1; d < 4; d *= 2) {
    l_a += __shfl_xor_sync(0xffffffffu, l_a, d);
    l_b += __shfl_xor_sync(0xffffffffu, l_b, d);
  }
  if ((lane & 3) == 0) {
    s_m[warp][ra] = m_a;
    s_m[warp][rb] = m_b;
    s_l[warp][ra] = l_a;
    s_l[warp][rb] = l_b;
  }
  if (tid < kTileRows) s_odd[tid] = 0;
  __syncthreads();  // every ring is free
  float* part = reinterpret_cast<float*>(smem);  // [warp][row][D]
  static_assert(S::kWarps * kTileRows * D * 4 <= S::kRingBytes, "parts fit in the rings");
#pragma unroll
  for (int d = 0; d < ND; ++d) {
    const int at = d * 8 + (lane & 3) * 2;
    *reinterpret_cast<float2*>(part + (warp * kTileRows + ra) * D + at) = make_float2(o[d][0], o[d][1]);
    *reinterpret_cast<float2*>(part + (warp * kTileRows + rb) * D + at) = make_float2(o[d][2], o[d][3]);
  }
  __syncthreads();
  // the CTA's sums take the place of warp 0's part
  for (int i = tid; i < rows * (D / 4); i += NT) {
    const int row = i / (D / 4), c = i % (D / 4);
    float m = neg_inf();
#pragma unroll
    for (int k = 0; k < S::kWarps; ++k) m = fmaxf(m, s_m[k][row]);
    const float ref = m == neg_inf() ? 0.f : m;
    float l = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < S::kWarps; ++k) {
      const float w = exp2f(s_m[k][row] - ref);
      l += w * s_l[k][row];
      const float4 v = *reinterpret_cast<const float4*>(part + (k * kTileRows + row) * D + c * 4);
      sum.x = fmaf(w, v.x, sum.x);
      sum.y = fmaf(w, v.y, sum.y);
      sum.z = fmaf(w, v.z, sum.z);
      sum.w = fmaf(w, v.w, sum.w);
    }
    *reinterpret_cast<float4*>(part + row * D + c * 4) = sum;
    if (c == 0) {
      s_cta_m[row] = m;
      s_cta_l[row] = l;
    }
    if (!(finite(sum.x) && finite(sum.y) && finite(sum.z) && finite(sum.w) && finite(l))) s_odd[row] = 1;
  }
  __syncthreads();
  for (int row = warp; row < rows; row += S::kWarps) {
    const int32_t lim = row_limit(a, rq, token_of(row));
    if (!s_odd[row] || lim >= hi) continue;
    // keys past the row's limit were in its tiles
    float m, l, x[D / 32];
    row_by_keys<D>(a, r, h, a.q.data + int64_t(rq.tok0 + token_of(row)) * a.q.ts + head_of(row) * a.q.hs, lo, lim, m, l,
                   x);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) part[row * D + lane + 32 * i] = x[i];
    if (lane == 0) {
      s_cta_m[row] = m;
      s_cta_l[row] = l;
    }
  }

  // ---- join the splits' sums, and the parts of the grid before: each CTA of
  // the cluster a share of the rows' vectors, read from all of them
  if (a.splits > 1) cluster_sync();
  else __syncthreads();
  wait_for_previous();
  const int64_t part_rows = int64_t(a.num_tokens) * a.num_heads;
  const uint32_t part_at = smem_addr(part), m_at = smem_addr(s_cta_m), l_at = smem_addr(s_cta_l);
  for (int i = split * NT + tid; i < rows * (D / 4); i += NT * a.splits) {
    const int row = i / (D / 4), c = i % (D / 4);
    const int64_t t = rq.tok0 + token_of(row);
    const int32_t head = head_of(row);
    const int64_t part_row = t * a.num_heads + head;
    float m = neg_inf();
    for (int k = 0; k < a.splits; ++k) m = fmaxf(m, ld_cluster(in_cta(m_at + row * 4, k)));
    for (int k = 0; k < a.num_parts; ++k) m = fmaxf(m, __ldcg(&a.part_ml[k * part_rows + part_row].x));
    const float ref = m == neg_inf() ? 0.f : m;
    float l = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < a.splits; ++k) {
      const float w = exp2f(ld_cluster(in_cta(m_at + row * 4, k)) - ref);
      l += w * ld_cluster(in_cta(l_at + row * 4, k));
      const float4 v = ld_cluster4(in_cta(part_at + (row * D + c * 4) * 4, k));
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
      const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + (k * part_rows + part_row) * D + c * 4));
      sum.x = fmaf(w, v.x, sum.x);
      sum.y = fmaf(w, v.y, sum.y);
      sum.z = fmaf(w, v.z, sum.z);
      sum.w = fmaf(w, v.w, sum.w);
    }
    // a sum of 0: no key was seen, or none with a score above -inf
    const bool none = l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
    if (none) sum = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<uint2*>(a.out.data + t * a.out.ts + head * a.out.hs + c * 4) =
        make_uint2(to_bf16x2(sum.x * inv, sum.y * inv), to_bf16x2(sum.z * inv, sum.w * inv));
    if (a.lse != nullptr && c == 0)
      a.lse[part_row] = none ? neg_inf() : (m + log2f(l)) * kLn2;
  }
  if (s_failed && tid == 0) record(a.st, kErrTimeout, r);
  if (a.splits > 1) cluster_sync();  // no CTA leaves while another reads it
}

}  // namespace isq
