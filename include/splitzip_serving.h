/*
 * splitzip_serving.h -- the operators around a KV cache, next to the codec of
 * splitzip.h that packs and sends it: what fills the cache, what reads it, how
 * much attention its tokens got, and what thins it before it is sent.
 *
 *   splitzip_qk_norm_rope       per-head RMS norm of queries and keys and the
 *                               position rotation in one pass, keys and values
 *                               stored into the cache by slot
 *   splitzip_attention          softmax attention over the cache: causal, with
 *                               an optional sliding window and a few first
 *                               tokens that stay visible (sinks); whole
 *                               prompts, chunks and single tokens
 *   splitzip_attention_weights  the softmax weight each cached token gets from
 *                               given queries, summed over them
 *   splitzip_evict              keep the first, the last and the most attended
 *                               tokens of a cache, in order, in a smaller one
 *
 * A cache is any strided view [batch, tokens, kv_heads, head_dim] of BF16 or
 * FP8 E5M2 values; in the layout [layers, 2, tokens, kv_heads, head_dim] that
 * the codec's callers use, keys and values of one layer or of all layers
 * (batch = layers) are such views without a copy.
 *
 * Ownership, streams and errors are those of splitzip.h: the library allocates
 * nothing, every device pointer is caller-owned memory on the current device,
 * every call only enqueues on the caller's stream, a failed host-side check
 * returns SPLITZIP_ERR_INVALID_ARG and enqueues nothing, a CUDA failure
 * returns SPLITZIP_ERR_CUDA.  Lengths, slots and positions that live in device
 * memory are checked where they are used, so no value of theirs makes a call
 * read or write outside the given buffers.  The outputs of a call may not
 * overlap its inputs except where a call says so.
 */
#ifndef SPLITZIP_SERVING_H
#define SPLITZIP_SERVING_H

#include "splitzip.h"
#include "splitzip_transfer.h" /* SPLITZIP_FORMAT_BF16, SPLITZIP_FORMAT_E5M2 */

#ifdef __cplusplus
extern "C" {
#endif

/* A strided view [batch, tokens, heads, head_dim]: the head_dim values of a row
 * contiguous, `data` and all strides (counted in elements) multiples of 16
 * bytes, strides positive and below 2^38; stride_b of an input may be 0 (one
 * sequence shared by the batch).  Strides of dimensions of length 1 are not
 * looked at, nor stride_b where a call takes no batch. */
typedef struct splitzip_view {
    void *data;
    int64_t stride_b, stride_t, stride_h;
} splitzip_view;

/* Query heads per key/value head that the attention calls accept. */
#define SPLITZIP_MAX_GROUP 64u

/* ------------------------------------------- norm, rotation, cache write */

/* For each of n tokens: q_out = rotate(norm(q) * q_weight) for every query
 * head, k_cache[slot] = rotate(norm(k) * k_weight) and v_cache[slot] = v for
 * every key/value head, with norm(x) = x / sqrt(mean(x^2) + eps).
 * The rotation turns the first rot_dim values of a head by the angles of the
 * token's position: pairs (i, i + rot_dim/2), or (2i, 2i+1) if interleaved,
 * become (a c - b s, b c + a s) with c = table[pos][i], s = table[pos][rot_dim/2 + i].
 * Arithmetic is in 32 bits, with one rounding to the stored type (to nearest
 * even; E5M2 values past the largest finite one become infinite).
 *   q, k, v        BF16 [n, heads, head_dim], e.g. slices of a fused projection
 *   q_weight, k_weight  head_dim BF16 values (16-byte aligned), or NULL for 1
 *   positions      int32[n] (may be NULL if rot_dim is 0); a token whose
 *                  position is outside [0, table_rows) gets NaN in the
 *                  rotated values of its queries and keys
 *   table          float[table_rows][rot_dim], 16-byte aligned
 *   slots          int64[n]: the cache row, counted in stride_t steps from
 *                  `data`, each used once; a token whose slot is outside
 *                  [0, cache_rows), or in a gap of the cache, writes its
 *                  queries only
 *   q_out          BF16 [n, q_heads, head_dim]; may be q itself
 *   k_cache, v_cache  rows [cache_rows, kv_heads, head_dim] of cache_format
 *   cache_step, cache_tokens  0, or the caches hold sequences with gaps between
 *                  them: sequence b's token t is row b * cache_step + t, and
 *                  rows from cache_tokens on to the next sequence's first are
 *                  no part of the caches; cache_rows is then at most 2^32
 * head_dim 64 or 128; rot_dim a multiple of 8 up to head_dim, or 0;
 * n * (q_heads + 2 kv_heads) < 2^31.  One launch; n = 0 enqueues nothing. */
typedef struct splitzip_norm_rope_args {
    splitzip_view q, k, v;
    const void *q_weight, *k_weight;
    const int32_t *positions;
    const float *table;
    const int64_t *slots;
    splitzip_view q_out, k_cache, v_cache;
    uint64_t table_rows, cache_rows;
    uint32_t n, q_heads, kv_heads, head_dim, rot_dim;
    uint32_t cache_format; /* SPLITZIP_FORMAT_BF16 or SPLITZIP_FORMAT_E5M2 */
    uint32_t interleaved;
    float eps; /* >= 0 */
    uint32_t cache_step, cache_tokens;
} splitzip_norm_rope_args;

splitzip_status splitzip_qk_norm_rope(const splitzip_norm_rope_args *args, splitzip_stream_t s);

/* ------------------------------------------------------------- attention */

/* What attention and its weights share.  Sequence b holds lens[b] tokens
 * (clamped to [0, kv_tokens]; kv_tokens if lens is NULL), the last q_tokens of
 * which are its queries: query i is at position p = lens[b] - q_tokens + i and
 * sees slot t if t <= p and (window = 0 or t > p - window or t < sinks).  A
 * shorter sequence in a batch simply has its queries right-aligned; a query at
 * a negative position sees nothing.  Slots that a query does not see
 * contribute nothing to it, whatever they hold (NaN and infinities too).
 * Query head h reads key/value head h / (q_heads / kv_heads).
 *   q     BF16 [batch, q_tokens, q_heads, head_dim]
 *   k, v  [batch, kv_tokens, kv_heads, head_dim] of cache_format
 * head_dim 64 or 128; q_heads a multiple of kv_heads, at most
 * SPLITZIP_MAX_GROUP times it.  q_tokens * (q_heads / kv_heads) and kv_tokens
 * at most 2^31 - 256, batch * kv_heads < 2^31. */
typedef struct splitzip_attention_args {
    splitzip_view q, k, v;
    splitzip_view out;   /* BF16 like q (attention only) */
    float *lse;          /* float[batch][q_heads][q_tokens]: attention's output
                            (may be NULL), attention_weights' input */
    const int32_t *lens; /* int32[batch] or NULL */
    uint32_t batch, q_tokens, kv_tokens, q_heads, kv_heads, head_dim;
    uint32_t window, sinks;
    uint32_t cache_format;
    float scale;         /* of the scores, finite */
} splitzip_attention_args;

/* Bytes of workspace splitzip_attention needs for these sizes (views, lens and
 * scale are not looked at); zero-filled once after allocation
 * (splitzip_workspace_init), kept consistent by the calls, shared by calls
 * that are ordered on one stream and need no more than it holds.  0 for sizes
 * that are refused. */
size_t splitzip_attention_workspace_bytes(const splitzip_attention_args *args);

/* out = softmax(scale q k^T over the visible slots) v, and lse = log(sum
 * exp(scale q k^T)) (natural logarithm).  A query that sees nothing, or scores
 * of -infinity alone, gets out = 0 and lse = -inf, and gives no weight below.
 * Scores, the softmax statistics and sums are held in 32 bits.  A weight counts
 * for out in 16 bits, as its product with the values takes it: BF16 over BF16
 * caches (off by up to 2^-8 of itself), FP16 over E5M2 (2^-11, below 2^-22 of the
 * row's largest by up to 2^-33 of that), where queries too are FP16, of their row
 * scaled by a power of two.  workspace:
 * 16-byte aligned, workspace_bytes of it. */
splitzip_status splitzip_attention(const splitzip_attention_args *args, void *workspace,
                                   size_t workspace_bytes, splitzip_stream_t s);

/* Synchronise s and report on the calls of splitzip_attention that ran on this
 * workspace since the last report: SPLITZIP_OK, or SPLITZIP_ERR_TIMEOUT if a
 * bounded wait inside a kernel gave up (its rows of out and lse are NaN).  The
 * workspace stays usable. */
splitzip_status splitzip_attention_status(void *workspace, splitzip_stream_t s);

/* weights_out[b][h][t] = weights_in[b][h][t] + the sum over the queries i and
 * the query heads of key/value head h that see slot t of
 * exp(scale q.k - lse): the softmax weight the slot got from them.  A sum's
 * order is fixed.  lse comes from splitzip_attention with the same mask, and q
 * may be any of its queries (with lens and q_tokens placing them);
 * q.k of a masked slot is not looked at.  Both float[batch][kv_heads][kv_tokens];
 * weights_in may be weights_out, or NULL for zeros.  Slots past a sequence's
 * length get weights_in.  Needs no workspace; v and out are ignored.  If a bounded wait
 * inside the kernel gives up, the weights it had not finished are NaN. */
splitzip_status splitzip_attention_weights(const splitzip_attention_args *args,
                                           const float *weights_in, float *weights_out,
                                           splitzip_stream_t s);

/* -------------------------------------------------------------- eviction */

/* Thin every (sequence, key/value head) of a cache to at most `budget` slots.
 * With n = lens[b] (clamped to [0, kv_tokens]; kv_tokens if NULL): if n <=
 * budget all n are kept, else slots below keep_first, slots from n - keep_last
 * on, and of the others the budget - keep_first - keep_last with the largest
 * weights (of equal weights the lower slot; NaN counts as the smallest).
 * Kept slots stay in order: index[b][h][j] is the old slot of new slot j, and
 * k_out / v_out [batch, budget, kv_heads, head_dim] and weights_out its rows
 * and weight.  New slots from min(n, budget) on get index -1, zero rows and
 * weight 0.
 *   weights      float[batch][kv_heads][kv_tokens], as
 *                splitzip_attention_weights accumulates them
 *   index        int32[batch][kv_heads][budget]
 *   weights_out  float[batch][kv_heads][budget], may be NULL
 *   lens_out     int32[batch], min(n, budget), may be NULL
 * keep_first + keep_last <= budget; budget >= 1; head_dim 64 or 128;
 * batch <= 65535; kv_tokens, batch * kv_heads < 2^31; budget * kv_heads <
 * 2^35.  Two launches. */
typedef struct splitzip_evict_args {
    splitzip_view k, v, k_out, v_out;
    const float *weights;
    const int32_t *lens;
    int32_t *index;
    float *weights_out;
    int32_t *lens_out;
    uint32_t batch, kv_tokens, kv_heads, head_dim, budget;
    uint32_t keep_first, keep_last;
    uint32_t cache_format;
} splitzip_evict_args;

splitzip_status splitzip_evict(const splitzip_evict_args *args, splitzip_stream_t s);

#ifdef __cplusplus
}
#endif

#endif /* SPLITZIP_SERVING_H */
