/*
 * inject_query.h -- C-ABI of the query side: what a serving engine runs, per
 * layer, after is_inject_batch has put a request's facts into the paged KV
 * cache and only the query tokens are left to prefill or decode.
 *
 *   is_query_rotate   per-head RMS norm (optional) and RoPE rotation of
 *                     queries and keys, one pass over both;
 *   is_query_append   keys (normed, rotated) and values of new tokens written
 *                     to their slots of the paged cache, the queries rotated
 *                     in the same launch;
 *   is_query_attend   attention of the query tokens over the paged cache,
 *                     with a prefix shared by the whole batch.
 *
 * Conventions as in inject_store.h: bf16 tensors as void*, IS_OK or a
 * negative IS_ERR_* status, no call aborts the process or takes ownership of
 * a caller array, `stream` is a cudaStream_t of the handle's device, and the
 * work is asynchronous on it.  Device-side problems are recorded on the
 * device and returned by is_query_last_error.  The calls that launch work
 * allocate nothing, wait for nothing and may be captured into a CUDA graph.
 * A handle's calls may run at the same time on several streams (they share
 * only the status word, of which the first error is kept); the arrays that
 * two of them write must be distinct.  Handles are not internally locked:
 * create and destroy belong to one thread.
 */
#ifndef INJECT_QUERY_H
#define INJECT_QUERY_H

#include <stdint.h>

#include "inject_store.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct is_query is_query_t; /* opaque; owned by the library */

/* Create a query handle on `device`: the RoPE frequency table (fp64) and a
 * status word.  Of cfg it reads num_layers, num_kv_heads, head_dim (32, 64,
 * 128 or 256) and the RoPE fields, with is_store_create's meaning and
 * checks; the capacity, batch-limit and tier fields are ignored.  A store
 * with the same RoPE fields injects keys that these calls' keys agree with.
 * Errors: INVALID_ARG, NOT_SUPPORTED (head_dim), OOM, CUDA. */
int is_query_create(const is_store_config_t* cfg, int device, is_query_t** out);

/* Free the handle.  Waits for its device's work.  NULL is ignored. */
void is_query_destroy(is_query_t* query);

/* Wait for `stream`, then return and clear the first device-side error
 * recorded since the previous call (IS_OK if none); *detail_out, if not
 * NULL, receives its index (see each call).  Only `stream` is waited for: an
 * error of work that is still under way on another stream is kept for a later
 * call, one recorded there already is returned too.  A stream that is being
 * captured is refused (CUDA; the capture is lost). */
int is_query_last_error(is_query_t* query, void* stream, int64_t* detail_out);

/* Rows of head vectors: element (token t, head h, dim d) is
 * ((uint16_t*)data)[t*token_stride + h*head_stride + d].  Strides in
 * elements, multiples of 8; data 16-byte aligned.  A slice of a fused
 * projection's output is such rows.  A stride of 0 repeats a row of an input;
 * for rows that are written it is refused (INVALID_ARG). */
typedef struct {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
  int32_t num_heads;
} is_rows_t;

/* Norm and rotation of head vectors (head_dim D of the handle):
 *   n(x) = x * w / sqrt(mean(x^2) + eps)   with w bf16 [D], or x if w NULL
 *   y    = bf16_rne(R(positions[t]) n(x))
 * R is the RoPE rotation of the handle's configuration (fp64 angles, fp32
 * norm and rotation, one rounding).  q_out and k_out have their input's
 * number of heads and may be the input itself (same data and strides);
 * otherwise no output may overlap an input.  k (with k_out) may be NULL.
 *   positions   device int32 [num_tokens]; a negative one marks a padding
 *               token, whose rows are not written
 *   q_weight, k_weight   device bf16 [D], 16-byte aligned, or NULL
 *   eps         finite and >= 0, one for both
 * Errors: INVALID_ARG, CUDA.  num_tokens may be 0. */
int is_query_rotate(is_query_t* query, int32_t num_tokens, const int32_t* positions,
                    const is_rows_t* q, const is_rows_t* q_out, const void* q_weight,
                    const is_rows_t* k, const is_rows_t* k_out, const void* k_weight, float eps,
                    void* stream);

/* Append new tokens to the paged cache and rotate their queries:
 *   K cache row (layer, slots[t], head h) <- bf16_rne(R(positions[t]) n(k))
 *   V cache row (layer, slots[t], head h) <- v     (bit copy)
 *   q_out                                 <- as is_query_rotate (q not NULL)
 * k and v have the handle's num_kv_heads heads; cache is what
 * is_inject_batch takes, and slot s means block s / block_size, token
 * s % block_size of it, as in its slot mapping.
 *   slots       device int64 [num_tokens]; -1: the token's K and V are not
 *               stored (its queries are rotated all the same)
 *   positions   as above; a negative one skips the token whole
 * Tokens must not share slots (the winner is undefined).  No other cache
 * element is written.
 * Device-side error: BAD_BLOCK for a slot outside [-1, num_blocks *
 * block_size); that token's K and V are not stored, detail is the token.
 * Errors: INVALID_ARG, CUDA.  num_tokens may be 0. */
int is_query_append(is_query_t* query, int32_t num_tokens, const int32_t* positions,
                    const int64_t* slots, const is_rows_t* k, const is_rows_t* v,
                    const void* k_weight, const is_rows_t* q, const is_rows_t* q_out,
                    const void* q_weight, float eps, const is_cache_t* cache, int32_t layer,
                    void* stream);

/* One attention call.  Request r owns query tokens q_offsets[r] ..
 * q_offsets[r+1] (n_r of them); its query i stands at position
 * start_pos[r] + i and sees the keys of positions
 *   j < kv_lens[r], and with causal also j <= start_pos[r] + i.
 * Position j < shared_len lies in block shared_blocks[j / B], any other in
 * block_tables[r][j / B], at token j % B of it (a shared_len inside a block
 * is allowed: that block's first part comes from the shared list).  Query
 * head h reads KV head h / (num_q_heads / num_kv_heads):
 *   out[t][h] = bf16_rne(sum_j p_j v_j),  p = softmax_j(scale q . k_j)
 * in fp32.  The probabilities meet v as sums of two bf16 values, within 2^-16
 * of them, for up to 16 rows (max_q_len queries x query heads of a KV head) and
 * with head_dim 256; for more rows with head_dim 32, 64 or 128 rounded to bf16.
 * A query that sees no key, or none with a score above -inf, gets zeros and
 * lse -inf.  NaN and infinities in cache elements that a query does not see do
 * not reach it (its sum may then run in another order). */
typedef struct {
  int32_t num_tokens;            /* rows of q, out and lse                     */
  int32_t num_requests;
  int32_t max_q_len;             /* >= every n_r (decides the launch shape)    */
  int32_t max_blocks_per_req;    /* row length of block_tables (bounds the keys
                                    and so decides the launch shape: rows far
                                    wider than the lengths cost a few requests
                                    some 4 us for a second grid)               */
  const int32_t* q_offsets;      /* device [num_requests + 1], non-decreasing  */
  const int32_t* start_pos;      /* device [num_requests]                      */
  const int32_t* kv_lens;        /* device [num_requests]                      */
  const int32_t* block_tables;   /* device [num_requests][max_blocks_per_req]; a
                                    row's entries below shared_len / B and from
                                    kv_lens[r] on are not read                 */
  const int32_t* shared_blocks;  /* device [ceil(shared_len / B)], or NULL     */
  int32_t shared_len;            /* >= 0; 0: no shared prefix                  */
  int32_t causal;                /* 0 or 1                                     */
  float scale;                   /* > 0; 0: 1 / sqrt(head_dim)                 */
  int32_t layer;
  is_rows_t q;                   /* num_heads a multiple of num_kv_heads       */
  is_rows_t out;                 /* q's number of heads; may be q itself       */
  float* lse;                    /* NULL, or device [num_tokens][heads]: natural
                                    log of the sum of exp(scale q . k_j)       */
} is_attend_t;

/* Bytes of device work space that is_query_attend needs for these arguments
 * (the arrays are not read; 0 is possible).  It depends on num_tokens,
 * num_requests, max_q_len, max_blocks_per_req, shared_len, the cache's block
 * size and q's number of heads alone.  Errors: INVALID_ARG, CAPACITY. */
int is_query_attend_workspace(const is_query_t* query, const is_attend_t* args,
                              const is_cache_t* cache, int64_t* bytes_out);

/* Run it.  workspace: device memory, 256-byte aligned, of at least the bytes
 * above (NULL if 0), written by this call alone until it has finished: two
 * calls in flight, or two graphs that may replay at the same time, need one
 * each.  Rows of out and lse behind q_offsets[num_requests] are left as they
 * were.
 * Device-side errors (the first recorded one is kept):
 *   INVALID_ARG  a request whose offsets decrease or leave [0, num_tokens],
 *                that has more than max_q_len queries, or a negative
 *                start_pos or kv_len (request skipped, detail: request)
 *   POSITION     kv_lens[r] past max_blocks_per_req * block_size and past
 *                shared_len, or above 2^31 - 129 (request skipped, detail:
 *                request)
 *   BAD_BLOCK    a block that is read lies outside [0, num_blocks): its
 *                keys are left out (detail: request, or -1 for a shared one)
 *   TIMEOUT      a wait inside a kernel gave up (seconds; a fault of the
 *                library, the call's rows are undefined)
 * A skipped request's rows are left as they were.  Requests whose token
 * ranges overlap (a decreasing offset elsewhere) have undefined rows.
 * Errors: INVALID_ARG, CAPACITY (workspace too small, more than 2^31 - 1
 * rows of num_tokens * heads, or shared_len above 2^31 - 129), CUDA. */
int is_query_attend(is_query_t* query, const is_attend_t* args, const is_cache_t* cache,
                    void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* INJECT_QUERY_H */
