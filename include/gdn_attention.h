/*
 * gdn_attention.h -- C ABI of rotary positions, of writing keys and values
 * into a paged cache, and of attention over that cache, on one GB300 GPU: what
 * the attention layers beside gated delta rule layers need, on the same packed
 * batches and on the pages of gdn_pages.h.
 *
 * Rotary positions.  Pair i of a head (i < R / 2, R = rotary_dim <= D) is
 * turned by the angle p * frequencies[i], p the token's position:
 *
 *     (a, b) -> magnitude * (a cos - b sin, b cos + a sin)
 *
 * with (a, b) = (x[i], x[i + R / 2]), or (x[2 i], x[2 i + 1]) when interleaved;
 * channels R .. D - 1 stay as they are.  The angle's fraction of a turn is
 * formed in integers, right to 2^-33 of a turn at positions as far as 2^31;
 * sines, products and sums are fp32, the result is rounded once.  The backward
 * pass is the same call with inverse != 0: the turn the other way.
 *
 * The cache.  A page is one row of k and of v, [n_pages, page_tokens, kv_heads,
 * D] with any strides over contiguous channels; table, lengths and n_pages are
 * those of gdn_pages.h.  A step brings n_i new tokens to sequence i of the
 * batch, which is row seqs[i] of the table; lengths[seqs[i]] counts the
 * sequence's tokens with the new ones, so new token j has position
 * p = lengths - n_i + j and lies in page table[seqs[i]][p / page_tokens].
 *
 * Attention.  New token j of head h sees the keys s of its sequence with
 *
 *     0 <= s < lengths,   s <= p (causal),   s > p - window (window > 0)
 *
 * and o = sum_s w_s v_s, w = softmax_s(scale q . k_s), with key head
 * h / (heads / kv_heads).  Scores, maxima, sums and o are fp32; with 16-bit
 * types the tensor cores take w relative to the row's running maximum rounded
 * to that type; o is rounded once.  lse = log sum_s exp(scale q . k_s).  A row
 * that sees nothing has o = 0 and lse = -infinity.  A key that a row does not
 * see has no influence on it, whatever it holds.  A channel in which a row sees
 * an infinite value is infinite; NaN, where it sees both signs or NaN, or where
 * that value's weight vanishes in its type.
 *
 * Shapes (device memory):
 *   q, q_out, output    [T, heads, D], k, v and k_out [T, kv_heads, D]: a
 *                       token's heads contiguous, *_stride elements from token
 *                       to token (0: dense)
 *   frequencies         [R / 2] double, radians a token
 *   positions           [T] int32 or int64
 *   cu_seqlens          [N + 1] int32 or int64: 0, non-decreasing, at most T;
 *                       rows past cu_seqlens[N] belong to nobody: append and
 *                       attention leave them as they were, gdn_rotary_run goes
 *                       on counting their positions
 *   seqs                [N] int32; NULL: sequence i is row i
 *   lse                 [T, heads] fp32, dense
 *
 * Ownership, streams and errors are those of gdn_prefill.h: the caller owns
 * every tensor and the workspace, runs only enqueue work on the caller's
 * stream, and what the host can check is refused before anything is launched.
 * What depends on device data sets bits of *device_status (optional):
 *   GDN_DEVICE_ERR_CU_SEQLENS  cu_seqlens out of order or past T
 *   GDN_PAGES_ERR_SEQ          a sequence outside [0, max_seqs): it has no
 *                              tokens in the cache
 *   GDN_PAGES_ERR_PAGE         a negative length (taken as 0), or one past the
 *                              table, or a page outside [0, n_pages): tokens
 *                              without a page are not written, and nobody sees
 *                              them
 *   GDN_DEVICE_ERR_TIMEOUT     a wait inside the attention kernel ran out; the
 *                              outputs are then NaN where they depend on it
 * Sequences of one append call have to differ; two that name one row race.
 */
#ifndef GDN_ATTENTION_H
#define GDN_ATTENTION_H

#include "gdn_pages.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ROTARY_MAX_DIM 1024   /* D of rotary calls */
#define GDN_ATTENTION_MAX_DIM 256 /* D of attention calls */
#define GDN_ATTENTION_MAX_TOKENS 0x7fff0000LL /* T of append and attention calls */

/* The new tokens of a step, and where they stand in the cache. */
typedef struct gdn_kv_batch {
    const void *cu_seqlens; /* NULL: every sequence has tokens_per_seq tokens */
    const int32_t *seqs;    /* NULL: sequence i is row i */
    const int32_t *table, *lengths;
    int64_t total_tokens; /* T */
    int32_t num_seqs;     /* N */
    int32_t tokens_per_seq;
    int32_t cu_i64;
    int32_t max_seqs, max_pages, n_pages, page_tokens;
    int32_t *device_status; /* optional */
} gdn_kv_batch;

/* Strides in elements; pages, tokens and heads do not overlap. */
typedef struct gdn_kv_cache {
    void *k, *v;
    int64_t k_page_stride, k_token_stride, k_head_stride;
    int64_t v_page_stride, v_token_stride, v_head_stride;
    int32_t kv_heads, head_dim;
    gdn_dtype dtype; /* BF16, F16 or F32; q, k, v and the outputs have it too */
} gdn_kv_cache;

/* What is turned, and how.  q or k may be NULL (heads or kv_heads 0). */
typedef struct gdn_rotary_args {
    const void *q, *k;
    void *q_out, *k_out; /* q and k themselves (same stride), or apart from q, k, v and each other */
    int64_t q_stride, k_stride, q_out_stride, k_out_stride;
    const double *frequencies;
    int32_t heads, kv_heads, head_dim, rotary_dim; /* rotary_dim even, 0 <= R <= D */
    int32_t interleaved, inverse;
    float magnitude;
    gdn_dtype dtype;
} gdn_rotary_args;

/* Positions are given, or count from 0 in every sequence of cu_seqlens, or
 * (both NULL) from 0 over all rows. */
gdn_status gdn_rotary_run(const gdn_rotary_args *args, const void *positions, int32_t positions_i64, const void *cu_seqlens,
                          int32_t cu_i64, int32_t num_seqs, int64_t total_tokens, void *stream);

/* k, turned, and v, as it is, into the cache; q, turned, to q_out (both NULL:
 * keys and values alone).  args' k_out is not used; rotary_dim = 0 turns
 * nothing.  v [T, kv_heads, D] has v_stride elements from token to token.  All
 * of them are apart from the caches, which is not checked. */
gdn_status gdn_cache_append_run(const gdn_kv_batch *batch, const gdn_kv_cache *cache, const gdn_rotary_args *args, const void *v,
                                int64_t v_stride, void *stream);

typedef struct gdn_attention_args {
    const void *q;
    void *output; /* its rows apart from q's */
    float *lse; /* optional; apart from q and output */
    int64_t q_stride, output_stride;
    int32_t heads;
    float scale;
    int32_t causal, window; /* window 0: none */
} gdn_attention_args;

/* Bytes of workspace (16-byte aligned device memory) that a run of these
 * arguments needs on the current device; 0 for arguments that it refuses.  A
 * workspace serves one run at a time. */
size_t gdn_attention_workspace(const gdn_kv_batch *batch, const gdn_kv_cache *cache, const gdn_attention_args *args);

gdn_status gdn_attention_run(const gdn_kv_batch *batch, const gdn_kv_cache *cache, const gdn_attention_args *args, void *workspace,
                             size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTENTION_H */
