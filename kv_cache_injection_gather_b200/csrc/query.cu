// Host side of the query calls declared in include/inject_query.h: the
// handle, the checks of arguments and the launches of the kernels in
// query_rows.cuh, attend_rows.cuh and attend_tiles.cuh.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <new>

#include "attend_rows.cuh"
#include "attend_tiles.cuh"
#include "inject_query.h"
#include "query_rows.cuh"

struct is_query {
  int device = 0;
  int sm_count = 148;
  int64_t clusters[4] = {};  // of 2^i CTAs of attend_rows that run at once; 0: none of this size
  int32_t num_layers = 0, kv_heads = 0, head_dim = 0, style = 0;
  double* turns = nullptr;  // [head_dim / 2] RoPE frequencies over 2 pi
  isq::Status* status = nullptr;
  std::mutex taking;         // one is_query_last_error at a time takes the status
  PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;  // the driver's
};

namespace {

struct OnDevice {
  int prev = -1;
  explicit OnDevice(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev) cudaSetDevice(dev);
    else prev = -1;
  }
  ~OnDevice() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

void free_query(is_query* q) {
  if (!q) return;
  cudaFree(q->turns);
  cudaFree(q->status);
  delete q;
}

// A failed runtime call's error is this call's: no later one finds it.
int cuda_error() {
  cudaGetLastError();
  return IS_ERR_CUDA;
}

// Launches; whether that worked is said by the launch alone.
template <typename... Args>
bool start(void (*fn)(Args...), unsigned grid, unsigned threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, fn, args...) == cudaSuccess;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Kernel tables over head_dim and its variants.
using RowsKernel = void (*)(isq::RowArgs);
template <int D>
RowsKernel rows_kernel_of(int style, bool norm) {
  if (style) return norm ? &isq::rows_kernel<D, 1, true> : &isq::rows_kernel<D, 1, false>;
  return norm ? &isq::rows_kernel<D, 0, true> : &isq::rows_kernel<D, 0, false>;
}
RowsKernel rows_kernel_of(int D, int style, bool norm) {
  switch (D) {
    case 32: return rows_kernel_of<32>(style, norm);
    case 64: return rows_kernel_of<64>(style, norm);
    case 128: return rows_kernel_of<128>(style, norm);
    case 256: return rows_kernel_of<256>(style, norm);
    default: return nullptr;
  }
}

struct AttendKernel {
  void (*fn)(isq::AttendArgs, CUtensorMap, CUtensorMap);
  int smem, threads, rows;  // rows of a unit
};
// The streaming kernel: units of 16 rows; of 32 for head_dim 32, whose long
// requests it takes too.
template <int D, int NR>
AttendKernel attend_rows_of() {
  return {&isq::attend_rows_kernel<D, NR>, isq::RowsShape<D, NR>::kSmemBytes, isq::RowsShape<D, NR>::kThreads, NR};
}
template <int D>
AttendKernel attend_rows_of(int64_t most) {
  return most <= 16 ? attend_rows_of<D, 16>() : attend_rows_of<D, 32>();
}
// For requests of up to `most` rows per KV head.
AttendKernel attend_rows_of(int D, int64_t most) {
  switch (D) {
    case 32: return attend_rows_of<32>(most);
    case 64: return attend_rows_of<64, 16>();
    case 128: return attend_rows_of<128, 16>();
    default: return attend_rows_of<256, 16>();
  }
}

// The kernel for many rows: head_dim 64 and 128 (fn is nullptr otherwise).
template <int D>
AttendKernel attend_tiles_of(bool shared) {
  return {shared ? &isq::attend_tiles_kernel<D, true> : &isq::attend_tiles_kernel<D, false>,
          isq::TilesShape<D>::kSmemBytes, isq::TilesShape<D>::kThreads, isq::kUnitRows};
}
AttendKernel attend_tiles_of(int D, bool shared) {
  if (D == 64) return attend_tiles_of<64>(shared);
  if (D == 128) return attend_tiles_of<128>(shared);
  return {nullptr, 0, 0, 0};
}
// What joins parts, of either kernel (head_dim 32 has none).
using JoinKernel = void (*)(isq::AttendArgs);
JoinKernel join_parts_of(int D) {
  switch (D) {
    case 64: return &isq::join_parts_kernel<64>;
    case 128: return &isq::join_parts_kernel<128>;
    case 256: return &isq::join_parts_kernel<256>;
    default: return nullptr;
  }
}

// Rows of a KV head and request up to which attend_rows takes them where
// attend_tiles could (64 requests of 2250 keys: 32 rows take 164 us against 139,
// 64 rows 272 against 141; attend_tiles costs as much for any number).
constexpr int kMostNarrowRows = 16;
// Keys that a split of a unit's keys should at least have, and a part.
constexpr int kKeysPerSplit = 128;
constexpr int kKeysPerPart = 512;
constexpr int kKeysPerRowPart = 256;
// Parts of attend_rows cost a grid more, some 4 us: taken where they spare a
// CTA this many keys of a cluster's split, more where the clusters are
// enough CTAs to fill the memory's bandwidth.
constexpr int kKeysSpared = 1536;
constexpr int kKeysSparedFull = 3000;
// The shared prefix gets a grid of its own (attend_tiles over all requests'
// rows) where the requests would otherwise read this many bytes of it.  Decode,
// 4 queries a KV head, 100 own keys; with this grid against without it, us:
//                 8 k shared                       131 k shared
//   KV heads      1        2        4        8     1        2        4         8
//   2 requests    -        -        -        -     97/31    102/43   105/66    116/114
//   8 requests    -      23/25    25/25    25/39  100/66   104/113   106/234   119/454
//   64 requests  35/39    37/66    48/127   71/248 158/453  160/891   177/1719  215/3394
// So bytes alone are too simple a rule for a few requests with few KV heads
// behind a very long prefix: kMostPrefixParts leaves SMs without work there, and
// the grid costs up to 3 times what the requests' own would.
constexpr int64_t kSharedBytes = 64 << 20;
// Its keys are split into parts of this many tiles, as few CTAs as that: they
// run beside the requests' grid, which is short of bandwidth and not of SMs
// (100 requests of 2000 keys behind 4096 shared: 171 us; with parts of 2 tiles,
// which take every SM first, 187; of 16, which end last, 192).  The requests'
// grid reads every part's sums again for each row, so they are kept few; other
// bounds than 16 were not measured.
constexpr int kTilesPerPart = 8;
constexpr int kMostPrefixParts = 16;
constexpr int kMostParts = 32;  // a lane each in join_parts
// A unit's tiles times its shares are counted in 32 bits (attend_tiles: parts;
// attend_rows: CTAs of a cluster times parts).
static_assert((int64_t(isq::kMostKeys) / isq::kTileKeys + 1) * std::max(kMostParts, kMostPrefixParts) * isq::kMostSplits <=
                  int64_t(1) << 32,
              "tile numbers");

// Fills in the clusters of 2^i CTAs that run at once, as ask(CTAs, number)
// says: one CTA an SM, but a cluster's in one GPC, so a part of a GPU may have
// room for none of the larger ones.  False where not even one CTA runs.
template <typename Ask>
bool count_clusters(int64_t (&clusters)[4], Ask ask) {
  for (int i = 0; i < 4; ++i) {
    int n = 0;
    if (ask(1u << i, &n) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    clusters[i] = n;
  }
  return clusters[0] > 0;
}

// What an attention call launches; all from the host's numbers.
struct AttendPlan {
  bool wide;             // attend_tiles over requests, else attend_rows
  bool shared;           // before it, attend_tiles over the shared prefix
  AttendKernel kernel;   // of the requests
  int64_t units;         // of the requests' grid
  int32_t splits;        // of attend_rows (a cluster)
  int32_t key_parts;     // of attend_rows, that a grid behind joins; 1: none
  int32_t parts;         // in the work space: of the prefix, or of the requests' keys; 0: none
  int64_t shared_units;
  int64_t ml_bytes, o_bytes;  // work space
};

int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

AttendPlan plan_attend(const is_query* q, const is_attend_t* a, const is_cache_t* c) {
  AttendPlan p{};
  const int64_t group = a->q.num_heads / q->kv_heads;
  const int64_t rows = int64_t(a->num_tokens) * group;
  const int64_t most = int64_t(std::min(a->max_q_len, a->num_tokens)) * group;
  const int64_t keys = std::max<int64_t>(int64_t(a->max_blocks_per_req) * c->block_size, a->shared_len);
  const bool has_tiles = attend_tiles_of(q->head_dim, false).fn != nullptr;
  p.wide = has_tiles && most > kMostNarrowRows;
  p.kernel = p.wide ? attend_tiles_of(q->head_dim, false) : attend_rows_of(q->head_dim, most);
  const int64_t unit_rows = p.kernel.rows;
  // one unit per request where it holds all the request's rows, else at most
  // a partial unit per request more than the rows fill
  p.units = most <= unit_rows ? a->num_requests : (rows + unit_rows - 1) / unit_rows + a->num_requests;
  const int64_t ctas = p.units * q->kv_heads;
  p.splits = p.key_parts = 1;
  if (p.wide) {
    // few CTAs: the keys of each in parts, that a grid behind joins
    const int64_t most_parts = std::min<int64_t>({q->sm_count / ctas, keys / kKeysPerPart, kMostParts});
    if (most_parts > 1) p.parts = int32_t(most_parts);
  } else {
    const int64_t prefix = int64_t(a->shared_len) * a->num_requests * q->kv_heads * q->head_dim * 4;
    p.shared = has_tiles && a->num_requests > 1 && prefix >= kSharedBytes;
    if (p.shared) {
      p.shared_units = (rows + isq::kUnitRows - 1) / isq::kUnitRows;
      const int64_t most_parts = q->sm_count / (p.shared_units * q->kv_heads);
      const int64_t tiles = (int64_t(a->shared_len) + isq::kTileKeys - 1) / isq::kTileKeys;
      p.parts = int32_t(std::max<int64_t>(
          1, std::min<int64_t>({most_parts, (tiles + kTilesPerPart - 1) / kTilesPerPart, kMostPrefixParts})));
    }
    // The keys of a unit are split over a cluster while all clusters run at
    // once (a CTA has an SM to itself and costs some 10 000 cycles of start and
    // end: 10 requests of 2250 keys take 31 us so, and 41 with twice the CTAs).
    const int64_t own = keys - (p.shared ? a->shared_len : 0);
    for (int i = 1; (1 << i) <= isq::kMostSplits && ctas <= q->clusters[i] && own >= (kKeysPerSplit << i); ++i)
      p.splits = 1 << i;
    // Few units of many keys: shares for every SM, in clusters as small as
    // kMostParts allows (larger ones leave SMs unused), whose sums are parts
    // that a grid behind joins.  One decoding request of 131 k keys, 8 KV heads:
    // 117 us in clusters, 94 so; 1 KV head: 116 and 25; of 16 k keys, 8 heads: 25
    // and 27.
    const int64_t shares = std::min<int64_t>(q->sm_count / ctas, own / kKeysPerRowPart);
    const bool full = ctas * p.splits * 8 > int64_t(q->sm_count) * 5;
    if (!p.shared && shares > p.splits && join_parts_of(q->head_dim) &&
        own / p.splits - own / shares >= (full ? kKeysSparedFull : kKeysSpared)) {
      const int i = shares > 3 * kMostParts ? 2 : shares > kMostParts ? 1 : 0;
      const int64_t parts = std::min<int64_t>({kMostParts, shares >> i, q->clusters[i] / ctas});
      if (parts > 1) {
        p.splits = 1 << i;
        p.parts = p.key_parts = int32_t(parts);
      }
    }
  }
  if (p.parts) {
    const int64_t part_rows = int64_t(p.parts) * a->num_tokens * a->q.num_heads;
    p.ml_bytes = round256(part_rows * int64_t(sizeof(float2)));
    p.o_bytes = part_rows * q->head_dim * int64_t(sizeof(float));
  }
  return p;
}

// Rows as the kernels take them; false where the header's rules are broken.
bool rows_ok(const is_rows_t* r) {
  return r && r->data && aligned16(r->data) && r->num_heads > 0 && r->token_stride >= 0 && r->head_stride >= 0 &&
         r->token_stride % 8 == 0 && r->head_stride % 8 == 0;
}
// Rows that are written: no two at one place by a stride of 0.
bool out_ok(const is_rows_t* r, int32_t num_tokens) {
  return rows_ok(r) && (r->token_stride > 0 || num_tokens == 1) && (r->head_stride > 0 || r->num_heads == 1);
}
isq::Rows rows_of(const is_rows_t& r) {
  return {static_cast<uint16_t*>(r.data), r.token_stride, r.head_stride};
}

bool cache_ok(const is_query* q, const is_cache_t* c, int32_t layer) {
  return c && c->k_cache && c->v_cache && aligned16(c->k_cache) && aligned16(c->v_cache) && c->num_blocks > 0 &&
         c->block_size >= 1 && c->block_size <= 128 && layer >= 0 && layer < q->num_layers && c->layer_stride >= 0 &&
         c->block_stride >= 0 && c->token_stride >= 0 && c->head_stride >= 0 && c->layer_stride % 8 == 0 &&
         c->block_stride % 8 == 0 && c->token_stride % 8 == 0 && c->head_stride % 8 == 0;
}
uint16_t* layer_of(void* cache, const is_cache_t* c, int32_t layer) {
  return static_cast<uint16_t*>(cache) + int64_t(layer) * c->layer_stride;
}

// Tensor maps of a layer's K and V with the cache's strides, as [64 dims]
// [8 tokens][slabs of 64 dims][groups of 8 tokens][blocks] (32 dims for D =
// 32); the head is a slab number.  A box is a head's dims x the largest power
// of two of tokens that divides the block and a tile of keys.  Returns that
// power's logarithm, or -1 where there is no such box: under 8 tokens, a head
// stride between slabs, strides that a map cannot have, a driver that makes no
// maps (the kernels then gather key by key).
int box_maps(const is_query* q, isq::AttendArgs& a, CUtensorMap& k, CUtensorMap& v) {
  int box = 0;
  while ((2 << box) <= isq::kTileKeys && a.block_size % (2 << box) == 0) ++box;
  const int D = q->head_dim, slab = std::min(D, 64);
  const int64_t slabs = (a.kv_heads - 1) * (a.head_stride / slab) + D / slab;
  if (!q->encode || box < 3 || a.head_stride % slab != 0 || slabs > INT32_MAX) return -1;
  a.head_slabs = int32_t(a.kv_heads > 1 ? a.head_stride / slab : 0);
  const cuuint64_t dims[5] = {cuuint64_t(slab), 8, cuuint64_t(slabs), cuuint64_t(a.block_size / 8), cuuint64_t(a.num_blocks)};
  const cuuint64_t strides[4] = {cuuint64_t(a.token_stride) * 2, cuuint64_t(slab) * 2, cuuint64_t(a.token_stride) * 16,
                                 cuuint64_t(a.block_stride) * 2};
  const cuuint32_t boxes[5] = {cuuint32_t(slab), 8, cuuint32_t(D / slab), cuuint32_t(1 << box) / 8, 1};
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  const CUtensorMapSwizzle swizzle = slab == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  for (int i = 0; i < 2; ++i)
    if (q->encode(i ? &v : &k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<uint16_t*>(i ? a.v_cache : a.k_cache), dims,
                  strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return -1;
  return box;
}

int launch_rows(const is_query* q, const isq::RowArgs& a, int32_t num_tokens, cudaStream_t st) {
  const int64_t want = (int64_t(std::max({a.nq, a.nk, a.nv})) * (q->head_dim / 16) + 31) / 32 * 32;
  // Few tokens: a thread a row and role, for latency.  Many: 64 threads with
  // several rows each, whose loads are in flight together and which share a
  // token's angles (16384 tokens, 40 normed heads: 60 us, with 128 threads 72).
  const int most = num_tokens < 4 * q->sm_count ? isq::kRowThreads : 64;
  const bool norm = a.q_weight != nullptr || a.k_weight != nullptr;
  const unsigned threads = unsigned(std::min<int64_t>(want, most));
  return start(rows_kernel_of(q->head_dim, q->style, norm), unsigned(num_tokens), threads, st, a) ? IS_OK : cuda_error();
}

// The arguments of an attention call that do not need the device; IS_OK, or
// the error.
int check_attend(const is_query* q, const is_attend_t* a, const is_cache_t* c) {
  if (!q || !a || !cache_ok(q, c, a->layer)) return IS_ERR_INVALID_ARG;
  if (a->num_tokens < 0 || a->num_requests < 0 || a->max_q_len < 0 || a->max_blocks_per_req < 0 || a->shared_len < 0 ||
      (a->causal != 0 && a->causal != 1) || !(a->scale >= 0.f) || !std::isfinite(a->scale))
    return IS_ERR_INVALID_ARG;
  if (a->q.num_heads <= 0 || a->q.num_heads % q->kv_heads != 0 || a->out.num_heads != a->q.num_heads)
    return IS_ERR_INVALID_ARG;
  if (a->num_tokens > 0 && a->num_requests > 0) {
    if (!rows_ok(&a->q) || !out_ok(&a->out, a->num_tokens) || !a->q_offsets || !a->start_pos || !a->kv_lens ||
        a->max_q_len < 1 || (a->max_blocks_per_req > 0 && !a->block_tables) || (a->shared_len > 0 && !a->shared_blocks))
      return IS_ERR_INVALID_ARG;
  }
  if (int64_t(a->num_tokens) * a->q.num_heads > INT32_MAX || a->shared_len > isq::kMostKeys) return IS_ERR_CAPACITY;
  return IS_OK;
}

}  // namespace

extern "C" {

int is_query_create(const is_store_config_t* cfg, int device, is_query_t** out) {
  if (!cfg || !out) return IS_ERR_INVALID_ARG;
  *out = nullptr;
  const is_store_config_t& c = *cfg;
  if (c.num_layers < 1 || c.num_kv_heads < 1 || !(c.rope_theta > 0) ||
      (c.rope_style != IS_ROPE_ROTATE_HALF && c.rope_style != IS_ROPE_INTERLEAVED) ||
      (c.rope_scaling != IS_SCALING_NONE && c.rope_scaling != IS_SCALING_LLAMA3))
    return IS_ERR_INVALID_ARG;
  if (c.rope_scaling == IS_SCALING_LLAMA3 &&
      (!(c.scale_factor > 0) || !(c.low_freq_factor > 0) || !(c.high_freq_factor > c.low_freq_factor) ||
       c.original_max_position < 1))
    return IS_ERR_INVALID_ARG;
  if (!rows_kernel_of(c.head_dim, 0, false)) return IS_ERR_NOT_SUPPORTED;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || device < 0 || device >= ndev) return cuda_error();
  OnDevice guard(device);
  is_query* q = new (std::nothrow) is_query();
  if (!q) return IS_ERR_OOM;
  q->device = device;
  q->num_layers = c.num_layers;
  q->kv_heads = c.num_kv_heads;
  q->head_dim = c.head_dim;
  q->style = c.rope_style;
  cudaDeviceGetAttribute(&q->sm_count, cudaDevAttrMultiProcessorCount, device);
  if (cudaMalloc(reinterpret_cast<void**>(&q->turns), sizeof(double) * size_t(c.head_dim / 2)) != cudaSuccess ||
      cudaMalloc(reinterpret_cast<void**>(&q->status), sizeof(isq::Status)) != cudaSuccess) {
    cudaGetLastError();
    free_query(q);
    return IS_ERR_OOM;
  }
  // Attributes now, so that the calls are launches alone (the functions are
  // loaded here, not inside somebody's stream capture).
  cudaFuncAttributes attr;
  bool ok = cudaFuncGetAttributes(&attr, reinterpret_cast<const void*>(&isq::take_status_kernel)) == cudaSuccess;
  for (bool norm : {false, true})
    ok = ok && cudaFuncGetAttributes(&attr, reinterpret_cast<const void*>(
                                                rows_kernel_of(c.head_dim, c.rope_style, norm))) == cudaSuccess;
  if (join_parts_of(c.head_dim))
    ok = ok && cudaFuncGetAttributes(&attr, reinterpret_cast<const void*>(join_parts_of(c.head_dim))) == cudaSuccess;
  for (const AttendKernel& k : {attend_rows_of(c.head_dim, 16), attend_rows_of(c.head_dim, 32),
                                attend_tiles_of(c.head_dim, false), attend_tiles_of(c.head_dim, true)})
    ok = ok && (!k.fn || cudaFuncSetAttribute(reinterpret_cast<const void*>(k.fn),
                                              cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem) == cudaSuccess);
  ok = ok && count_clusters(q->clusters, [&](unsigned ctas, int* n) {
         const AttendKernel k = attend_rows_of(c.head_dim, 16);
         cudaLaunchAttribute size{};
         size.id = cudaLaunchAttributeClusterDimension;
         size.val.clusterDim = {ctas, 1, 1};
         cudaLaunchConfig_t one{};
         one.gridDim = dim3(ctas);
         one.blockDim = dim3(unsigned(k.threads));
         one.dynamicSmemBytes = size_t(k.smem);
         one.attrs = &size;
         one.numAttrs = 1;
         return cudaOccupancyMaxActiveClusters(n, k.fn, &one);
       });
  void* encode = nullptr;
  cudaDriverEntryPointQueryResult found{};
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &encode, 12000, cudaEnableDefault, &found) ==
          cudaSuccess &&
      found == cudaDriverEntryPointSuccess)
    q->encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(encode);
  ok = ok && cudaMemset(q->status, 0, sizeof(isq::Status)) == cudaSuccess;
  ok = ok && start(&isq::turns_kernel, unsigned(c.head_dim / 2 + 127) / 128, 128, nullptr, q->turns, int(c.head_dim),
                   c.rope_theta, int(c.rope_scaling), c.scale_factor, c.low_freq_factor, c.high_freq_factor,
                   double(c.original_max_position));
  if (!ok || cudaDeviceSynchronize() != cudaSuccess) {
    free_query(q);
    return cuda_error();
  }
  *out = q;
  return IS_OK;
}

void is_query_destroy(is_query_t* q) {
  if (!q) return;
  OnDevice guard(q->device);
  cudaDeviceSynchronize();
  free_query(q);
}

int is_query_last_error(is_query_t* q, void* stream, int64_t* detail) {
  if (!q) return IS_ERR_INVALID_ARG;
  OnDevice guard(q->device);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Its work is done first, so that nothing is waited for under the lock (and
  // a stream that is being captured is refused before a launch).
  if (cudaStreamSynchronize(st) != cudaSuccess) return cuda_error();
  std::lock_guard<std::mutex> lock(q->taking);
  unsigned long long word = 0;
  if (!start(&isq::take_status_kernel, 1, 1, st, q->status) ||
      cudaMemcpyAsync(&word, &q->status->taken, sizeof(word), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return cuda_error();
  if (detail) *detail = int32_t(uint32_t(word));
  return int32_t(uint32_t(word >> 32));
}

int is_query_rotate(is_query_t* query, int32_t num_tokens, const int32_t* positions, const is_rows_t* q,
                    const is_rows_t* q_out, const void* q_weight, const is_rows_t* k, const is_rows_t* k_out,
                    const void* k_weight, float eps, void* stream) {
  if (!query || num_tokens < 0 || !(eps >= 0.f) || !std::isfinite(eps)) return IS_ERR_INVALID_ARG;
  if (num_tokens == 0) return IS_OK;
  if (!positions || !rows_ok(q) || !out_ok(q_out, num_tokens) || q->num_heads != q_out->num_heads ||
      !aligned16(q_weight) || !aligned16(k_weight) || (k == nullptr) != (k_out == nullptr))
    return IS_ERR_INVALID_ARG;
  if (k && (!rows_ok(k) || !out_ok(k_out, num_tokens) || k->num_heads != k_out->num_heads)) return IS_ERR_INVALID_ARG;
  OnDevice guard(query->device);
  isq::RowArgs a{};
  a.positions = positions;
  a.nq = q->num_heads;
  a.q = rows_of(*q);
  a.q_out = rows_of(*q_out);
  a.q_weight = static_cast<const uint16_t*>(q_weight);
  if (k) {
    a.nk = k->num_heads;
    a.k = rows_of(*k);
    a.k_out = rows_of(*k_out);
    a.k_weight = static_cast<const uint16_t*>(k_weight);
  }
  a.eps = eps;
  a.turns = query->turns;
  a.st = query->status;
  return launch_rows(query, a, num_tokens, static_cast<cudaStream_t>(stream));
}

int is_query_append(is_query_t* query, int32_t num_tokens, const int32_t* positions, const int64_t* slots,
                    const is_rows_t* k, const is_rows_t* v, const void* k_weight, const is_rows_t* q,
                    const is_rows_t* q_out, const void* q_weight, float eps, const is_cache_t* cache, int32_t layer,
                    void* stream) {
  if (!query || num_tokens < 0 || !(eps >= 0.f) || !std::isfinite(eps) || !cache_ok(query, cache, layer))
    return IS_ERR_INVALID_ARG;
  if (num_tokens == 0) return IS_OK;
  if (!positions || !slots || !rows_ok(k) || !rows_ok(v) || k->num_heads != query->kv_heads ||
      v->num_heads != query->kv_heads || !aligned16(k_weight) || !aligned16(q_weight) ||
      (q == nullptr) != (q_out == nullptr))
    return IS_ERR_INVALID_ARG;
  if (q && (!rows_ok(q) || !out_ok(q_out, num_tokens) || q->num_heads != q_out->num_heads)) return IS_ERR_INVALID_ARG;
  OnDevice guard(query->device);
  isq::RowArgs a{};
  a.positions = positions;
  a.slots = slots;
  if (q) {
    a.nq = q->num_heads;
    a.q = rows_of(*q);
    a.q_out = rows_of(*q_out);
    a.q_weight = static_cast<const uint16_t*>(q_weight);
  }
  a.nk = a.nv = query->kv_heads;
  a.k = rows_of(*k);
  a.v = rows_of(*v);
  a.k_weight = static_cast<const uint16_t*>(k_weight);
  a.eps = eps;
  a.turns = query->turns;
  a.k_cache = layer_of(cache->k_cache, cache, layer);
  a.v_cache = layer_of(cache->v_cache, cache, layer);
  a.block_stride = cache->block_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.num_slots = int64_t(cache->num_blocks) * cache->block_size;
  a.block_size = cache->block_size;
  a.st = query->status;
  return launch_rows(query, a, num_tokens, static_cast<cudaStream_t>(stream));
}

int is_query_attend_workspace(const is_query_t* query, const is_attend_t* args, const is_cache_t* cache,
                              int64_t* bytes_out) {
  if (!bytes_out) return IS_ERR_INVALID_ARG;
  *bytes_out = 0;
  const int rc = check_attend(query, args, cache);
  if (rc != IS_OK) return rc;
  if (args->num_tokens > 0 && args->num_requests > 0) {
    const AttendPlan p = plan_attend(query, args, cache);
    *bytes_out = p.ml_bytes + p.o_bytes;
  }
  return IS_OK;
}

int is_query_attend(is_query_t* query, const is_attend_t* args, const is_cache_t* cache, void* workspace,
                    int64_t workspace_bytes, void* stream) {
  const int rc = check_attend(query, args, cache);
  if (rc != IS_OK) return rc;
  if (args->num_tokens == 0 || args->num_requests == 0) return IS_OK;
  const AttendPlan p = plan_attend(query, args, cache);
  if (p.ml_bytes + p.o_bytes > 0) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)) return IS_ERR_INVALID_ARG;
    if (workspace_bytes < p.ml_bytes + p.o_bytes) return IS_ERR_CAPACITY;
  }
  // attend_tiles: one dimension; attend_rows: (head, split), units, more units
  const int64_t shared_grid = p.shared_units * query->kv_heads * p.parts;
  const int64_t grid_x = query->kv_heads * (p.wide ? p.units * std::max(1, p.parts) : int64_t(p.key_parts) * p.splits) +
                         (p.wide ? 1 : 0);
  const int64_t grid_y = p.wide ? 1 : std::min<int64_t>(p.units + 1, 32768);
  const int64_t grid_z = p.wide ? 1 : (p.units + grid_y) / grid_y;
  if (grid_x > INT32_MAX || shared_grid > INT32_MAX || grid_z > 65535) return IS_ERR_CAPACITY;
  OnDevice guard(query->device);
  isq::AttendArgs a{};
  a.num_tokens = args->num_tokens;
  a.num_requests = args->num_requests;
  a.max_q_len = std::min(args->max_q_len, args->num_tokens);
  a.max_blocks = args->max_blocks_per_req;
  a.q_offsets = args->q_offsets;
  a.start_pos = args->start_pos;
  a.kv_lens = args->kv_lens;
  a.block_tables = args->block_tables;
  a.shared_blocks = args->shared_blocks;
  a.shared_len = a.table_shared = args->shared_len;
  a.causal = args->causal;
  const double scale = args->scale > 0.f ? double(args->scale) : 1.0 / std::sqrt(double(query->head_dim));
  a.scale_log2 = float(scale * 1.4426950408889634);
  a.num_heads = args->q.num_heads;
  a.kv_heads = query->kv_heads;
  a.group = a.num_heads / a.kv_heads;
  a.q = rows_of(args->q);
  a.out = rows_of(args->out);
  a.lse = args->lse;
  a.k_cache = layer_of(cache->k_cache, cache, args->layer);
  a.v_cache = layer_of(cache->v_cache, cache, args->layer);
  a.block_stride = cache->block_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.num_blocks = cache->num_blocks;
  a.block_size = cache->block_size;
  a.st = query->status;

  CUtensorMap k_map{}, v_map{};
  a.box_log2 = box_maps(query, a, k_map, v_map);
  if (p.parts) {
    a.part_ml = static_cast<float2*>(workspace);
    a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.ml_bytes);
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  auto launch = [&](const AttendKernel& k, dim3 grid) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(k.threads));
    cfg.dynamicSmemBytes = size_t(k.smem);
    return cudaLaunchKernelEx(&cfg, k.fn, a, k_map, v_map) == cudaSuccess;
  };
  // a grid that starts beside the one before it and waits for it at its end
  auto beside = [&] {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  };
  bool ok = true;
  if (p.shared) {
    a.splits = p.parts;
    a.units = p.shared_units;
    ok = launch(attend_tiles_of(query->head_dim, true), dim3(unsigned(shared_grid)));
    beside();
    a.num_parts = p.parts;
    a.first_key = a.shared_len;
    a.table_shared = 0;  // what is left of a request is in its own blocks
  }
  a.units = p.units;
  a.splits = p.wide ? std::max(1, p.parts) : p.splits;
  a.key_parts = p.key_parts;
  if (!p.wide && p.splits > 1) {
    while ((1 << a.splits_log2) < p.splits) ++a.splits_log2;
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs++].val.clusterDim = {unsigned(p.splits), 1, 1};
  }
  ok = ok && launch(p.kernel, dim3(unsigned(grid_x), unsigned(grid_y), unsigned(grid_z)));
  if (p.parts && !p.shared) {
    a.num_parts = p.parts;
    cfg.numAttrs = 0;
    beside();
    const int64_t rows = int64_t(a.num_tokens) * a.num_heads;
    cfg.gridDim = dim3(unsigned((rows + isq::kJoinRows - 1) / isq::kJoinRows));
    cfg.blockDim = dim3(isq::kJoinRows * 32);
    cfg.dynamicSmemBytes = 0;
    ok = ok && cudaLaunchKernelEx(&cfg, join_parts_of(query->head_dim), a) == cudaSuccess;
  }
  return ok ? IS_OK : cuda_error();
}

}  // extern "C"
