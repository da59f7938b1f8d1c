/*
 * mla_cache.h — C ABI of the calls that put tokens into the paged latent
 * cache (libmla_decode.so): rotary positions, and the append that norms the
 * latent, turns the RoPE dims and writes the row.
 *
 * The cache row is the one mla_decode reads ("DeepSeek V3/R1 Inference
 * Efficiency (2): Reverse-Engineering the Production Deployment", §2.4.1,
 * Compute: c + r = 512 + 64 dims a token; "How DeepSeek Inference Works",
 * levers table, "KV-cache layout (MLA, paging)"): 512 latent dims, 64 RoPE
 * dims, bf16 or FP8 (MLA_FP8_ROW_BYTES), in 64-token pages behind a block
 * table.
 *
 * Rotation: pair i of the R rotated dims of a row at position p is turned by
 * the angle p * inv_freq[i] and multiplied by `scale`:
 *
 *     (a, b) -> scale * (a cos - b sin, a sin + b cos)
 *
 * The pair is (2i, 2i + 1) (interleaved, the default) or (i, i + R / 2)
 * (MLA_FLAG_ROPE_HALF).  Scaling for long contexts is in inv_freq, which the
 * caller computes once (linear interpolation, YaRN, ...).  A factor that YaRN
 * puts on queries and keys may be `scale` only where every dim of a head turns;
 * with 64 of 192 it belongs, squared, into the attention's softmax_scale.
 * Frequencies are radians per position in fp64, of magnitudes below 2^52; the
 * angle is reduced modulo one turn in 64-bit fixed point, so that it is as exact
 * at position 2^31 - 1 as at 0 (off by 2^-32 turns at most, before its cosine
 * and sine are taken in fp32).
 *
 * Conventions: as for mla_decode.h (device pointers, asynchronous on
 * `stream`, no allocation, no host synchronisation, graph-capturable,
 * thread-safe).  Activations, weights and bf16 caches are 16-byte aligned,
 * strides are in elements and multiples of 8.
 */
#ifndef MLA_CACHE_H_
#define MLA_CACHE_H_

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  MLA_FLAG_ROPE_HALF = 32,    /* pairs (i, i + R / 2) instead of (2i, 2i + 1) */
  MLA_FLAG_ROPE_INVERSE = 64, /* the angle's sign is turned: the inverse rotation
                                 (with scale 1), and the rotation's gradient */
  MLA_MAX_ROPE_DIM = 256
};

/* Rotary positions over part of each head.
 *   x            bf16, row (t, h) at x + t * x_token_stride + h * x_head_stride,
 *                head_dim dims
 *   positions    int32 [num_tokens], any value
 *   num_heads    >= 1
 *   head_dim     multiple of 8; dims [rope_offset, rope_offset + rope_dim) are
 *                turned, the others copied
 *   rope_offset  multiple of 8
 *   rope_dim     multiple of 16, at most MLA_MAX_ROPE_DIM
 *   inv_freq     fp64 [rope_dim / 2], radians per position, below 2^52, 8-byte
 *                aligned
 *   scale        factor on the turned dims (finite)
 *   flags        MLA_FLAG_ROPE_HALF, MLA_FLAG_ROPE_INVERSE
 *   out          bf16, rows as x with its own strides; may be x itself with
 *                x's strides (in place), and must not overlap it otherwise
 * Products and sums are fp32, rounded to bf16 once. */
int mla_rope(const void* x, int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions,
             int num_tokens, int num_heads, int head_dim, int rope_offset, int rope_dim, const double* inv_freq,
             float scale, unsigned flags, void* out, int64_t out_token_stride, int64_t out_head_stride,
             mla_stream_t stream);

/* Append tokens to the paged latent cache.
 *   latent       bf16, row t at latent + t * latent_stride, 512 dims
 *   k_pe         bf16, row t at k_pe + t * k_pe_stride, 64 dims (a projection
 *                output [T, 576] is latent = base, k_pe = base + 512, both
 *                strides 576)
 *   norm_weight  bf16 [512] or NULL.  With it the stored latent is
 *                latent * norm_weight / sqrt(mean(latent^2) + eps)
 *   eps          >= 0, used with norm_weight only
 *   inv_freq     fp64 [32], below 2^52, or NULL (k_pe is stored as it is)
 *   rope_scale   factor on the turned dims (with inv_freq only)
 *   positions    int32 [num_tokens]: token t's position in its request's
 *                sequence, which is also its angle's; a negative position
 *                marks padding: nothing is read or written for that token
 *   request_ids  int32 [num_tokens] or NULL: token t's request.  NULL: the
 *                tokens are num_requests equal runs in order (num_tokens must
 *                be a multiple of num_requests)
 *   block_table, bt_stride, num_requests: as for mla_decode (rows of
 *                num_requests requests, bt_stride entries apart)
 *   bt_width     entries of a row that may be read, 1 .. bt_stride: a position
 *                must lie below 64 * bt_width
 *   kv_cache     bf16 [num_pages, 64, 576], or with MLA_FLAG_KV_FP8 bytes
 *                [num_pages, 64, 656]
 *   flags        MLA_FLAG_KV_FP8, MLA_FLAG_ROPE_HALF
 *   status       device int, set (from 0, atomically) to MLA_ERR_BAD_TABLE
 *                when a token's request, position or page is out of range;
 *                that token is skipped.  Never cleared by the call.
 * Every other row of the cache is left as it was.  No two tokens may name the
 * same row (which of them it then holds is not defined, and it may mix them).
 * The latent is normed in fp32 (its squares may leave fp32's range) and rounded
 * once, to bf16 or to E4M3.  An FP8 group of 128 dims takes the smallest
 * power-of-two scale that brings its largest finite magnitude to at most 448
 * (scale 1 for a group of zeros, and no scale below 2^-127); dims that are not
 * finite become NaN codes; the row's 12 unused bytes are written as zeros. */
int mla_cache_append(const void* latent, int64_t latent_stride, const void* k_pe, int64_t k_pe_stride,
                     const void* norm_weight, float eps, const double* inv_freq, float rope_scale,
                     const int32_t* positions, const int32_t* request_ids, int num_tokens,
                     const int32_t* block_table, int64_t bt_stride, int bt_width, int num_requests, void* kv_cache,
                     int64_t num_pages, unsigned flags, int* status, mla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_CACHE_H_ */
