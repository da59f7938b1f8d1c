/*
 * mla_prefix.h — C ABI of attention for a batch that shares a long prefix
 * (libmla_decode.so): the prefix's cached latents are expanded once into
 * per-head keys and values, and every step's query tokens attend to them in
 * one call, joined with what each request attends to on its own.
 *
 * The two forms of one attention ("DeepSeek V3/R1 Inference Efficiency (2):
 * Reverse-Engineering the Production Deployment", §2.4.1, Compute): absorbed,
 * a head scores the 576 dims of a cached row and sums its 512 latent dims,
 * 2 * (576 + 512) operations a (token, head, row), reading 1,152 bytes a row;
 * expanded, K[h] = W_UK[h]^T latent and V[h] = W_UV[h]^T latent of 128 dims
 * each, 2 * (192 + 128) operations, reading 512 bytes a (head, row).  One
 * request alone is served better by the absorbed form; when many requests
 * share the rows, the expanded form does 3.4 times less work and its bytes
 * are read once for all of them.
 *
 *     K[h, p, d] = sum_c latent[p, c] * W_UK[h, c, d]
 *     V[h, p, d] = sum_c latent[p, c] * W_UV[h, c, d]
 *     s[t, h, p] = softmax_scale * (q_nope[t, h] . K[h, p] + q_pe[t, h] . k_pe[p])
 *     out[t, h]  = sum_p softmax(s)_p * V[h, p],  lse[t, h] = ln sum_p exp(s_p)
 *
 * out is in the head's 128 value dims: the dims mla_absorb_o maps the
 * absorbed attention's output to, so the two join there.
 *
 * Conventions: as for mla_absorb.h (device pointers, 16-byte aligned,
 * strides in elements and multiples of 8, asynchronous on `stream`, no
 * allocation, no host synchronisation, graph-capturable).  `status` is a
 * device int the kernels set (from 0, atomically); the calls never clear it;
 * mla_workspace_status() reads it.  mla_prefix_attend calls whose work overlaps
 * on the GPU need workspaces of their own.
 */
#ifndef MLA_PREFIX_H_
#define MLA_PREFIX_H_

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Keys and values of a shared prefix.
 *   kv_cache, num_pages  as for mla_decode (FP8 rows with MLA_FLAG_KV_FP8)
 *   block_table  int32 [ceil(prefix_len / 64)]: the prefix's pages in order.
 *                An entry outside the pool sets *status to MLA_ERR_BAD_TABLE;
 *                its rows are then not specified (no fault).
 *   prefix_len   tokens of the prefix, >= 0
 *   w_uk, w_uv   bf16 [num_heads, 512, 128], as for mla_absorb_q / _o
 *   num_heads    1 .. 128
 *   k_nope       bf16 [num_heads, head_rows, 128], rows 0 .. prefix_len - 1 of
 *                each head written, the others left as they were
 *   v            fp16, laid out as k_nope (fp16, as every value product of
 *                the library takes: 11 significant bits).  A key or value
 *                that is not finite after its rounding (values from 65,520 on
 *                are not) sets *status to MLA_ERR_VALUE_RANGE
 *   head_rows    rows between heads, >= prefix_len, at most 2^30
 *   k_pe         bf16 [prefix_len, 64]: the rows' RoPE dims, copied
 *   status       also MLA_ERR_TIMEOUT if a bounded wait runs out
 * Sums are fp32, rounded once. */
int mla_prefix_expand(const void* kv_cache, int64_t num_pages, const int32_t* block_table, int prefix_len,
                      const void* w_uk, const void* w_uv, int num_heads, unsigned flags, void* k_nope, void* v,
                      int64_t head_rows, void* k_pe, int* status, mla_stream_t stream);

/* Bytes of workspace mla_prefix_attend needs on the current device, 0 where no
 * head's rows are split over SMs; 0 and *err set on failure (err may be NULL).
 * Host-only. */
size_t mla_prefix_attend_workspace_size(int num_tokens, int num_heads, int prefix_len, int* err);

/* Attention of num_tokens query tokens over one prefix.
 *   q_nope, q_pe bf16, row (t, h) at + (t * num_heads + h) * q_stride, 128 and
 *                64 dims (with the usual [T, H, 192] projection output, q_nope
 *                = base, q_pe = base + 128, q_stride = 192); q_pe already turned
 *   k_nope, v, head_rows, k_pe, prefix_len, num_heads: as mla_prefix_expand
 *                wrote them.  Every value of the prefix must be finite: a
 *                value row that is not reaches every token of the call that
 *                sees any row.  (Scores of rows that a token does not see may
 *                overflow.)
 *   visible      int32 [num_tokens] or NULL: token t sees the prefix's first
 *                visible[t] rows (clamped to 0 .. prefix_len): requests that
 *                share only part of it, and padded tokens (0).  NULL: all.
 *   softmax_scale  finite, > 0
 *   suffix_out, suffix_lse  both or neither: what each (token, head) attended
 *                to elsewhere, bf16 [num_tokens, num_heads, 128] and fp32
 *                [num_tokens, num_heads] natural log (-inf: nothing; the row
 *                of suffix_out is then not read as a number).  The result is
 *                the attention over both sets of rows.
 *   flags        MLA_FLAG_OUT_FP32
 *   out          [num_tokens, num_heads, 128] bf16 (fp32); may be suffix_out
 *                itself where both are bf16
 *   lse          fp32 [num_tokens, num_heads]; may be suffix_lse itself
 *   workspace    256-byte aligned, mla_prefix_attend_workspace_size bytes;
 *                NULL where none is needed
 *   status       MLA_ERR_TIMEOUT if a bounded wait runs out
 * A token that sees nothing, here and in the suffix, gets out = 0 and lse =
 * -inf.  Weights are exp in fp32, rounded to fp16 for the value product and
 * normalised by the sum of the rounded ones; sums are fp32. */
int mla_prefix_attend(const void* q_nope, const void* q_pe, int64_t q_stride, const void* k_nope, const void* v,
                      int64_t head_rows, const void* k_pe, int prefix_len, const int32_t* visible, int num_tokens,
                      int num_heads, float softmax_scale, const void* suffix_out, const float* suffix_lse,
                      unsigned flags, void* workspace, size_t ws_bytes, void* out, float* lse, int* status,
                      mla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_PREFIX_H_ */
