/*
 * mla_chunk.h — C ABI of attention for a chunk of new tokens over the paged
 * latent cache (libmla_decode.so): prompts that enter in chunks, the next
 * turns of conversations, draft trees longer than a decode step takes.
 *
 * Every request b of the batch has its own number of new tokens, n_b =
 * token_starts[b + 1] - token_starts[b], laid end to end in `q`; its cache
 * holds cache_lens[b] rows, the new tokens' own among them (mla_cache_append
 * comes first).  With MLA_FLAG_CAUSAL token i of request b sees the first
 * cache_lens[b] - n_b + i + 1 rows, else all cache_lens[b].  Over the V rows
 * that a token sees, per head,
 *
 *     s_j = softmax_scale * q . row_j          (576 dims)
 *     lse = ln sum_j exp(s_j),   out = sum_j exp(s_j - lse) * row_j[0 .. 511]
 *
 * and out = 0, lse = -inf where it sees none: mla_decode's attention, for any
 * number of tokens a request.
 *
 * Two tokens of a request share every tile of rows (the kernel of mla_decode's
 * two-token step), so a chunk costs 2 * 128 * 1088 operations a (token, row):
 * the right form up to some 160 tokens a request.  Beyond, and where the
 * memory is there, mla_prefix_expand followed by mla_prefix_attend with
 * `visible` counts does with less (8192 rows, absorptions included: 128 tokens
 * 232 us against 271, 160 289 / 289, 256 428 / 298).
 *
 * A request's odd token, and so a single one, costs what a pair does.  63
 * requests of one token over 4096 rows take 129 us (mla_decode with s_q = 1:
 * 114); beside 512 tokens of another request, in one call, 510 us (412 for those
 * alone, so that two calls are no faster).
 *
 * An FP8 cache's rows are widened to bf16 before, those of every request up to
 * its length, whatever the number of its tokens: 64 requests of 4 tokens over
 * 8192 rows take 574 us (bf16 rows 420; mla_decode 1,113, whose steps read FP8
 * rows once a token).
 *
 * Conventions: as for mla_decode.h (device pointers, asynchronous on `stream`,
 * no allocation, no host synchronisation, graph-capturable).
 */
#ifndef MLA_CHUNK_H_
#define MLA_CHUNK_H_

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace for a call of `num_tokens` tokens of `num_requests`
 * requests; `max_len` and `flags` as for the call (an FP8 cache's rows are
 * widened there once: num_requests * max_len rows of 1,152 bytes, 9.7 GB for 64
 * requests of up to 131,072 rows: give the longest length there is, and split a
 * batch over several calls where that is too much).  0 and *err (may be NULL) on
 * failure. */
size_t mla_chunk_attend_workspace_size(int num_tokens, int num_requests, int max_len, unsigned flags, int* err);

/*
 *   q             bf16 [num_tokens, 128, 576], contiguous, 16-B aligned
 *   kv_cache, num_pages: as for mla_decode (FP8 rows with MLA_FLAG_KV_FP8)
 *   block_table   int32, row b at block_table + b * bt_stride, of which the
 *                 first ceil(max_len / 64) entries may be read
 *   cache_lens    int32 [num_requests]
 *   max_len       an upper bound of every cache_lens[b] (<= 64 * bt_stride
 *                 where there is more than one request)
 *   token_starts  int32 [num_requests + 1], increasing from 0 or more to
 *                 num_tokens or less, or NULL: equal runs of num_tokens /
 *                 num_requests tokens.  Tokens of no request are left as they
 *                 were
 *   num_heads     must be 128
 *   flags         MLA_FLAG_CAUSAL, MLA_FLAG_OUT_FP32, MLA_FLAG_KV_FP8
 *   workspace     mla_chunk_attend_workspace_size bytes, 256-B aligned; a call
 *                 needs nothing of what an earlier one left there, and two
 *                 calls that may overlap need one each
 *   out           [num_tokens, 128, 512], bf16 (or fp32 with OUT_FP32); must
 *                 not overlap q
 *   lse           fp32 [num_tokens, 128], natural log
 *   status        device int, set (from 0, never cleared) to
 *                 MLA_ERR_BAD_TABLE if a length, a page (its rows read as
 *                 zeros) or a start is out of range, MLA_ERR_TIMEOUT if a
 *                 device wait ran out
 * A call without tokens looks at nothing and leaves `status` as it was.
 * Values have to stay below 65504 in magnitude (the value product is fp16, as
 * in mla_decode); rows that no token of a call sees may hold anything.
 */
int mla_chunk_attend(const void* q, const void* kv_cache, int64_t num_pages, const int32_t* block_table,
                     int64_t bt_stride, const int32_t* cache_lens, int max_len, const int32_t* token_starts,
                     int num_requests, int num_tokens, int num_heads, float softmax_scale, unsigned flags,
                     void* workspace, size_t ws_bytes, void* out, float* lse, int* status, mla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_CHUNK_H_ */
