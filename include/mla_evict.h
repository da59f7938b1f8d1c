/*
 * mla_evict.h — C ABI of what shrinks a cache by what was attended to
 * (libmla_decode.so): the attention weight that every cached row received,
 * the choice of the rows to keep, and their move to pages of their own.
 *
 * Conventions: as for mla_decode.h (device pointers, asynchronous on `stream`,
 * no allocation, no host synchronisation, graph-capturable).  `status` is a
 * device int that the kernels set (from 0, never cleared) to
 * MLA_ERR_BAD_TABLE if a length, a page or a start is out of range,
 * MLA_ERR_BAD_INDEX for a row outside its request, MLA_ERR_TIMEOUT if a
 * device wait ran out.
 */
#ifndef MLA_EVICT_H_
#define MLA_EVICT_H_

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace of mla_attention_weights; 0 and *err on failure. */
size_t mla_attention_weights_workspace_size(int num_tokens, int num_requests, int max_len, unsigned flags, int* err);

/*
 * What the query tokens of a step or a chunk attended to:
 *     out[b, j] = decay * weights[b, j] + sum_t sum_h exp(s[t, h, j] - lse[t, h])
 * over request b's tokens t that see row j, s as in mla_chunk.h.  Rows of
 * weights and out past cache_lens[b], and those of requests without tokens,
 * are left as they were.  The sum's order is fixed: equal calls give equal
 * bits.
 *   q, kv_cache, num_pages, block_table, bt_stride, cache_lens, max_len,
 *   token_starts, num_requests, num_tokens, num_heads, softmax_scale: as for
 *                 mla_chunk_attend
 *   lse           fp32 [num_tokens, 128], 16-B aligned: of the attention these are the
 *                 weights of (which may have seen more than this cache); -inf:
 *                 the head attended to nothing and adds nothing, whatever q
 *                 holds there
 *   weights, out  fp32 rows of max_len at a stride of weights_stride and
 *                 out_stride; out may be weights itself, and must not overlap
 *                 it otherwise.  weights may be NULL where decay is 0
 *   flags         MLA_FLAG_CAUSAL, MLA_FLAG_KV_FP8
 *   workspace     mla_attention_weights_workspace_size bytes, 256-B aligned;
 *                 two calls that may overlap need one each
 * A call without tokens looks at nothing and leaves `status` and `out` as they
 * were.
 */
int mla_attention_weights(const void* q, const float* lse, const void* kv_cache, int64_t num_pages,
                          const int32_t* block_table, int64_t bt_stride, const int32_t* cache_lens, int max_len,
                          const int32_t* token_starts, int num_requests, int num_tokens, int num_heads,
                          float softmax_scale, float decay, const float* weights, int64_t weights_stride,
                          unsigned flags, void* workspace, size_t ws_bytes, float* out, int64_t out_stride,
                          int* status, mla_stream_t stream);

/*
 * Which rows of each request stay: the first `sinks` and the last `recent`
 * ones, then those of the largest weight, of equal ones the first (+0 and -0
 * are equal; NaN counts as -inf), until there are min(cache_lens[b], keep).
 *   weights       fp32 [num_requests, max_len] at a stride of weights_stride
 *   cache_lens    int32 [num_requests], <= max_len
 *   keep          >= 1; 0 <= sinks, 0 <= recent, sinks + recent <= keep
 *   kept          int32 [num_requests, keep]: increasing positions, then -1
 *   new_lens      int32 [num_requests]; may be cache_lens itself, and must not
 *                 overlap it otherwise
 *   new_weights   fp32 [num_requests, new_width] at a stride of
 *                 new_weights_stride, new_width >= min(keep, max_len): the
 *                 kept rows' weights, then zeros; or NULL.  Must not overlap
 *                 weights
 */
int mla_evict_select(const float* weights, int64_t weights_stride, const int32_t* cache_lens, int num_requests,
                     int max_len, int keep, int sinks, int recent, int32_t* kept, int32_t* new_lens,
                     float* new_weights, int64_t new_weights_stride, int new_width, int* status,
                     mla_stream_t stream);

/*
 * Copies the kept rows to the pages of another table, in order: row kept[b, i]
 * of request b, at block_table[b][kept / 64], becomes row i at
 * out_table[b][i / 64], i < lens[b].  No page of out_table may hold a row that
 * kept names (pages of other requests included).
 *   cache         [num_pages, 64, row_bytes], 16-B aligned: the latent cache
 *                 (row_bytes 1152; FP8 656) or the indexer's keys (256)
 *   kept          int32 rows of kept_width at a stride of kept_stride
 *   lens          int32 [num_requests], <= kept_width
 */
int mla_cache_compact(void* cache, int64_t num_pages, int row_bytes, const int32_t* block_table, int64_t bt_stride,
                      int bt_width, const int32_t* kept, int64_t kept_stride, int kept_width, const int32_t* lens,
                      int num_requests, const int32_t* out_table, int64_t out_stride, int out_width, int* status,
                      mla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_EVICT_H_ */
