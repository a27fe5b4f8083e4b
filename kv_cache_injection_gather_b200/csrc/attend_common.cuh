// What the attention kernels share: arguments, barriers, copies, tensor-core
// instructions, the batch's requests and the paged cache's addresses.
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
  int64_t units;               // attend_rows: units of its grid
  int32_t splits;              // CTAs that share a unit's keys; attend_rows: a
  int32_t splits_log2;         // cluster of 1, 2, 4 or 8
  // Parts of the rows' sums in the work space, each [num_tokens][num_heads]:
  // (maximum, sum) pairs and [D] sums of values, all fp32.  attend_tiles
  // writes part `split`, attend_rows with key_parts > 1 one for each of them;
  // attend_rows and join_parts read num_parts of them.
  float2* part_ml;
  float* part_o;
  int32_t num_parts;
  int32_t key_parts;           // attend_rows: clusters that share a unit's keys
  int32_t first_key;           // attend_rows: the keys below are in the parts
  int32_t table_shared;        // positions below are looked up in shared_blocks
  // Keys of one tensor-map box (a power of two that divides the block size and
  // the kernel's tile), as a logarithm; -1: gather by rows.
  int32_t box_log2;
  int32_t head_slabs;          // slabs of dims between the maps' KV heads
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

// ---------------------------------------------------------------- barriers

__device__ __forceinline__ void bar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ bool bar_done(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// The rest of a wait: gives up after about two seconds, or once another thread
// has; without a flag only the limit counts.
__device__ __forceinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, volatile int32_t* failed) {
  const long long began = clock64();
  while (!bar_done(bar, parity)) {
    if (failed != nullptr && *failed) return false;
    if (clock64() - began > (1ll << 32)) {
      if (failed != nullptr) *failed = 1;
      return false;
    }
  }
  return true;
}
// Waits until the phase of the given parity has completed, or returns false.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int32_t* failed) {
  const uint32_t addr = smem_addr(bar);
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (bar_done(addr, parity)) return true;
  return bar_wait_long(addr, parity, failed);
}

// True in one lane of a converged warp.  The compiler knows it for one lane, so
// copies and products issued under it need no loop over lanes for their
// uniform operands (a lane-by-lane issue took 85 cycles an instruction).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
// One arrival that also announces bytes.
__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
// A box of the paged cache to shared memory: all dims of one head (`slab`: its
// first slab's number), tokens from 8 * group of `block`.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int32_t slab, int32_t group,
                                         int32_t block, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %3, %4, %5, "
      "%6}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_addr(bar)), "r"(0), "r"(slab), "r"(group), "r"(block)
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

// ---------------------------------------------------------------- tcgen05

__device__ __forceinline__ void tmem_alloc(uint32_t* at, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The barrier gets one arrival when all products issued so far by this thread
// are done.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
// N columns of this thread's lane.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 16) {
    tmem_ld16(addr, r);
  } else {
#pragma unroll
    for (int i = 0; i < N / 32; ++i) tmem_ld32(addr + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(&r[32 * i]));
  }
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[N]) {
  if constexpr (N == 16) {
    tmem_st16(addr, r);
  } else {
#pragma unroll
    for (int i = 0; i < N / 32; ++i) tmem_st32(addr + 32 * i, *reinterpret_cast<const uint32_t(*)[32]>(&r[32 * i]));
  }
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand descriptor (version 1) of a tile_at<D> layout: 128-byte
// swizzle for slabs of 64 dims (layout 2), 64-byte for one of 32 (layout 4).
// lead: bytes between the slabs of a transposed operand.
template <int D>
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
  return uint64_t((addr & 0x3ffff) >> 4) | (uint64_t(lead >> 4) << 16) | (uint64_t(D * 16 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(D < 64 ? 4 : 2) << 61);
}
// Instruction descriptor: bf16 x bf16 -> fp32, M = 128.  An operand that is
// stored with its product dimension (keys) across rows is transposed.
__host__ __device__ constexpr uint32_t product(int N, bool a_transposed, bool b_transposed) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_transposed ? 1u << 15 : 0u) | (b_transposed ? 1u << 16 : 0u) |
         (uint32_t(N / 8) << 17) | (uint32_t(128 / 16) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
      : "memory");
}

// Largest of a warp's values (NaN left out).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Address of the same shared variable in another CTA of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster2(uint32_t addr, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

// ---------------------------------------------------------------- requests

struct Request {
  int32_t tok0, n;      // its query tokens
  int32_t start, kv;    // position of the first, keys in the cache
};

// Positions of a request: a tile more still counts in 31 bits.
constexpr int32_t kMostKeys = INT32_MAX - 128;

// Reads request r; 0, or the error that makes the batch skip it.
__device__ __forceinline__ int32_t read_request(const AttendArgs& a, int32_t r, Request& q) {
  const int32_t t0 = a.q_offsets[r], t1 = a.q_offsets[r + 1];
  q.start = a.start_pos[r];
  q.kv = a.kv_lens[r];
  q.tok0 = t0;
  q.n = t1 - t0;
  if (t0 < 0 || t1 < t0 || t1 > a.num_tokens || q.n > a.max_q_len || q.start < 0 || q.kv < 0)
    return kErrInvalidArg;
  if (q.kv > kMostKeys || (q.kv > a.shared_len && q.kv > int64_t(a.max_blocks) * a.block_size)) return kErrPosition;
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
__device__ __forceinline__ const int32_t* table_slot(const AttendArgs& a, int32_t r, int32_t j) {
  const int32_t jb = j / a.block_size;
  return j < a.table_shared ? a.shared_blocks + jb : a.block_tables + int64_t(r) * a.max_blocks + jb;
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
  return entry_offset(a, r, h, j, *table_slot(a, r, j));
}

// ---------------------------------------------------------------- tiles

constexpr int kTileKeys = 128;

// A tile of bf16 rows of D values: groups of 8 rows, in them slabs of 64 dims
// (one of 32 for D = 32), in them the rows, their 16-byte chunks permuted by
// the row's number (the 128- and the 64-byte swizzle).  It is what the tensor
// cores read in both directions and what a tensor-map box of 8 tokens x slabs
// x groups of 8 writes in one go.  Byte offset of chunk c of a row:
template <int D>
__device__ __forceinline__ uint32_t tile_at(int row, int c) {
  if constexpr (D < 64) return uint32_t(row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
  return uint32_t((row >> 3) * (D * 16) + (c >> 3) * 1024 + (row & 7) * 128 + (((c & 7) ^ (row & 7)) << 4));
}
constexpr int kSlabStep = 1024;  // bytes between the slabs of a group (D >= 64)
// Byte offset of 16 dims at 16 * k, for all rows (the start of a product's
// step along the dims).
template <int D>
__device__ __forceinline__ uint32_t dims_at(int k) {
  return uint32_t((k >> 2) * kSlabStep + (k & 3) * 32);
}

// Warp g of W brings every W-th of the tiles K0 V0 K1 V1 ... of keys [lo, hi)
// of request r and KV head h into a ring of NS slots of kTileKeys x D.  (A
// tile's look-ups, waits and copies take one warp some 2000 cycles, mostly
// latency, so whole tiles go to warps in turn.)  full[] and empty[] take one
// arrival.  A tile comes as boxes, or key by key (keys outside
// [first_key, hi) as zeros) where a box holds keys of two blocks and where
// there is no map; with ZERO_EDGE also values that run past hi.  Boxes leave
// keys outside the range as they find them.  A block outside the cache sets
// *bad, and its keys mean nothing.
template <int D, int NS, int W>
__device__ __forceinline__ void gather_tiles(const AttendArgs& a, const CUtensorMap* k_map, const CUtensorMap* v_map,
                                             int g, int32_t r, int32_t h, int32_t lo, int32_t hi, int32_t tiles,
                                             unsigned char* ring, uint64_t* full, uint64_t* empty, uint64_t* edge,
                                             volatile int32_t* failed, int32_t* bad) {
  constexpr int CPR = D / 8, kSlotBytes = kTileKeys * D * 2;
  // A warp may wait for tile u - NS to be read only when tile u - 2 NS has
  // been: a parity tells neighbouring phases apart, no more.  Either the warp
  // has waited for that one (a slot is always the same warp's), or it has seen
  // tile u - W - NS read, a later one of the same kind, and keys are read in
  // order, and values are.
  static_assert(W <= NS && (NS % W == 0 || (NS - W) % 2 == 0), "phases of a slot in turn");
  const int lane = threadIdx.x & 31;
  const int32_t bits = max(0, a.box_log2), boxes = kTileKeys >> bits;
  const bool whole = a.block_size == 1 << bits;  // a box is a block
  const int32_t slab = h * a.head_slabs;
  auto by_box = [&](int32_t j0) {
    const bool torn = j0 < a.table_shared && a.table_shared - j0 < kTileKeys && (a.table_shared & ((1 << bits) - 1)) != 0;
    return a.box_log2 >= 0 && !torn;
  };
  // Lane i looks up box i of this warp's next tile (position -1: none), a tile
  // ahead of the copies that need it.
  int32_t next_pos, next_token, next_entry;
  auto look_up = [&](int32_t t) {
    const int32_t j0 = lo + t * kTileKeys, key = lane << bits;
    next_pos = a.box_log2 >= 0 && t < tiles && lane < boxes && hi - j0 > key ? j0 + key : -1;
    const int32_t jb = next_pos < 0 ? 0 : whole ? next_pos >> bits : next_pos / a.block_size;
    next_token = whole ? 0 : next_pos - jb * a.block_size;
    const int32_t* from = a.q_offsets;  // (a load in every case: one under a condition would be waited for there)
    if (next_pos >= 0)
      from = next_pos < a.table_shared ? a.shared_blocks + jb : a.block_tables + int64_t(r) * a.max_blocks + jb;
    next_entry = *from;
  };
  look_up(g / 2);
  int32_t u = g;
  for (; u < 2 * tiles; u += W) {
    const int32_t j0 = lo + (u >> 1) * kTileKeys;
    const bool v = u & 1;
    const CUtensorMap* map = v ? v_map : k_map;
    const uint16_t* cache = v ? a.v_cache : a.k_cache;
    const int slot = u % NS;
    const uint32_t dst = smem_addr(ring + slot * kSlotBytes);
    const int32_t pos = next_pos, entry = next_entry, group = next_token >> 3;
    const bool boxed = by_box(j0), fine = entry >= 0 && entry < a.num_blocks;
    const uint32_t good = __ballot_sync(0xffffffffu, pos >= 0 && fine);
    if (pos >= 0 && !fine && boxed) {
      record(a.st, kErrBadBlock, pos < a.table_shared ? -1 : r);
      *bad = 1;
    }
    look_up((u + W) >> 1);
    // the whole warp goes on or stops
    if (u >= NS && !__all_sync(0xffffffffu, bar_wait(&empty[slot], ((u / NS) - 1) & 1, failed))) break;
    if (boxed) {
      const bool clear = edge != nullptr && v && hi - j0 < kTileKeys;  // the last tile
      uint64_t* landed = clear ? edge : &full[slot];
      if (elect_one()) bar_expect(landed, (uint32_t(__popc(good)) << bits) * (D * 2));
      for (int box = 0; box < boxes; box += 8) {
        int32_t at_block[8], at_group[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          at_block[i] = __shfl_sync(0xffffffffu, entry, box + i);
          at_group[i] = whole ? 0 : __shfl_sync(0xffffffffu, group, box + i);
        }
        if (elect_one()) {
          const uint32_t step = uint32_t(D * 2) << bits, to = dst + box * step;
          if (((good >> box) & 255u) == 255u) {  // all there, as in most tiles
#pragma unroll
            for (int i = 0; i < 8; ++i) copy_box(to + i * step, map, slab, at_group[i], at_block[i], landed);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if ((good >> (box + i)) & 1u) copy_box(to + i * step, map, slab, at_group[i], at_block[i], landed);
          }
        }
      }
      if (clear) {
        if (!__all_sync(0xffffffffu, bar_wait(edge, 0, failed))) break;
        for (int i = (hi - j0) * CPR + lane; i < kTileKeys * CPR; i += 32)
          *reinterpret_cast<uint4*>(ring + slot * kSlotBytes + tile_at<D>(i / CPR, i % CPR)) = make_uint4(0, 0, 0, 0);
        proxy_fence();
        __syncwarp();
        if (lane == 0) bar_arrive(&full[slot]);
      }
    } else {
      for (int first = 0; first < kTileKeys; first += 32) {
        const int32_t j = j0 + first + lane;
        int64_t at = -1;
        if (hi - j0 > first + lane && j >= a.first_key) {
          at = key_offset(a, r, h, j);
          if (at < 0) *bad = 1;
        }
#pragma unroll 4
        for (int n = 0; n < CPR; ++n) {
          const int e = n * 32 + lane, row = e / CPR, c = e % CPR;
          const int64_t from = __shfl_sync(0xffffffffu, at, row);
          cp_async16(dst + tile_at<D>(first + row, c), cache + (from < 0 ? 0 : from + c * 8), from < 0 ? 0 : 16);
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
      proxy_fence();
      __syncwarp();
      if (lane == 0) bar_arrive(&full[slot]);
    }
  }
  if (*failed)  // copies in flight: nothing may leave before they land
    for (int32_t i = max(g, u - NS); i < u; i += W) bar_wait(&full[i % NS], (i / NS) & 1, nullptr);
}

// Queries of `rows` rows to a tile, zeros up to `count`, by `threads` threads.
template <int D, typename Source>
__device__ __forceinline__ void load_queries(unsigned char* tile, int rows, int count, int thread, int threads,
                                             const uint16_t* any, Source source) {
  constexpr int CPR = D / 8;
  for (int i = thread; i < count * CPR; i += threads) {
    const int row = i / CPR, c = i % CPR;
    const bool live = row < rows;
    cp_async16(smem_addr(tile + tile_at<D>(row, c)), live ? source(row) + c * 8 : any, live ? 16 : 0);
  }
  cp_async_commit();
  cp_async_wait<0>();
  proxy_fence();
}

// One row (of a tile of queries in shared memory) over keys [lo, hi) by a
// warp, key after key in fp32: for rows whose tiled product came out infinite
// or NaN although keys that they do not see may have caused it (0 * NaN).  o:
// dims lane, lane + 32, ...
template <int D>
__device__ __forceinline__ void row_by_keys(const AttendArgs& a, int32_t r, int32_t h, const unsigned char* q_tile,
                                            int row, int32_t lo, int32_t hi, float& m, float& l, float (&o)[D / 32]) {
  const int lane = threadIdx.x & 31;
  float x[D / 32];
  m = neg_inf();
  l = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int d = lane + 32 * i;
    x[i] = lo_f(*reinterpret_cast<const uint16_t*>(q_tile + tile_at<D>(row, d >> 3) + (d & 7) * 2));
    o[i] = 0.f;
  }
  for (int32_t j = lo; j < hi; ++j) {
    const int64_t at = key_offset(a, r, h, j);
    if (at < 0) continue;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      s = fmaf(x[i], lo_f(a.k_cache[at + lane + 32 * i]), s);
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
      o[i] = o[i] * shrink + p * lo_f(a.v_cache[at + lane + 32 * i]);
  }
}

}  // namespace isq
