/*
 * splitzip_pages.h -- a KV cache in pages, next to the strided one of
 * splitzip_serving.h: what writes it, what reads it back, and the attention of
 * new tokens over it.
 *
 *   splitzip_pages_store      keys and values of new tokens into their slots of
 *                             a pool, as they are or quantised to 8 or 4 bits
 *   splitzip_pages_load       sequences out of their pages into a strided cache,
 *                             for instance for the codec of splitzip.h to send
 *   splitzip_paged_attention  softmax attention of a batch's new tokens (single
 *                             ones, chunks of prompts, or both) over their
 *                             sequences' pages
 *
 * A pool is `pages` pages of `page_tokens` slots; a sequence's token t lies in
 * slot t % page_tokens of the page that its row of a table names at
 * t / page_tokens.
 *
 * Ownership, streams and errors are those of splitzip_serving.h: caller-owned
 * memory on the current device, calls only enqueue on the caller's stream, a
 * failed host-side check returns SPLITZIP_ERR_INVALID_ARG and enqueues nothing.
 * Slots, page numbers, lengths and query ranges that live in device memory are
 * checked where they are used: no value of theirs makes a call read or write
 * outside the given buffers.  The outputs of a call may not overlap its inputs.
 */
#ifndef SPLITZIP_PAGES_H
#define SPLITZIP_PAGES_H

#include "splitzip_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Formats of a pool, besides SPLITZIP_FORMAT_BF16 and SPLITZIP_FORMAT_E5M2.  A
 * quantised row is head_dim codes and four exponent bytes, one for each block of
 * head_dim / 4 values.  An exponent byte e stands for 2^(e - 127), 0 for 0, 255
 * for NaN, and a value is its code's times that.
 *   INT8  a code is a byte, a signed integer in [-127, 127]
 *   E2M1  a code is half a byte (the lower half first): sign, two exponent bits,
 *         one mantissa bit, for 0, 0.5, 1, 1.5, 2, 3, 4, 6
 * The store takes the smallest power with which the block's largest magnitude
 * does not round past the largest code, from 2^-24 to 2^9 (INT8) or from 2^-23 to
 * 2^13 (E2M1), and rounds each value once, to nearest even; larger values become
 * the largest one (65024, 49152).  A block that holds an infinity or a NaN
 * becomes NaN (255, codes 0), one of zeros 0 (0, codes 0 or -0).  All such values
 * are exact in BF16 and in FP16. */
#define SPLITZIP_FORMAT_INT8 2u
#define SPLITZIP_FORMAT_E2M1 3u

/* Rows [pages, page_tokens, kv_heads] of keys or values.  A row's codes are
 * contiguous: 2 head_dim bytes of BF16, head_dim of E5M2 and INT8, head_dim / 2
 * of E2M1; `data` and its strides (in BF16 values, else in bytes) are multiples of
 * 16 bytes, positive and below 2^38.  A row's four exponent bytes are contiguous,
 * `exponents` and its strides (in bytes) multiples of 4, positive and below 2^38;
 * NULL for BF16 and E5M2.  Strides of dimensions of length 1 are not looked at. */
typedef struct splitzip_page_rows {
    void *data;
    int64_t stride_p, stride_t, stride_h;
    uint8_t *exponents;
    int64_t exp_stride_p, exp_stride_t, exp_stride_h;
} splitzip_page_rows;

/* page_tokens a power of two from 16 to 65536; head_dim 64 or 128; pages < 2^31. */
typedef struct splitzip_pool {
    splitzip_page_rows k, v;
    uint32_t pages, page_tokens, kv_heads, head_dim, format;
} splitzip_pool;

/* ------------------------------------------------------------------ store */

/* The keys and values of n tokens into their slots.
 *   k, v   BF16 [n, kv_heads, head_dim], e.g. slices of a fused projection
 *   slots  int64[n], page * page_tokens + slot, each used once (a slot named twice
 *          holds a mixture of both tokens); a token whose slot is outside the pool
 *          is dropped
 * BF16 rows are copied, E5M2 values rounded to nearest even (infinite past the
 * largest finite one).  n * kv_heads < 2^31.  One launch; n = 0 enqueues nothing. */
typedef struct splitzip_pages_store_args {
    splitzip_view k, v;
    const int64_t *slots;
    splitzip_pool pool;
    uint32_t n;
} splitzip_pages_store_args;

splitzip_status splitzip_pages_store(const splitzip_pages_store_args *args, splitzip_stream_t s);

/* ------------------------------------------------------------------- load */

/* The first lens[b] (clamped to [0, tokens]; tokens if NULL) tokens of each
 * sequence out of their pages; rows behind them stay as they were.
 *   table         int32[batch][table_width]; entries that no token needs are not
 *                 looked at; a token whose page is outside the pool gives NaN
 *   k_out, v_out  [batch, tokens, kv_heads, head_dim] of out_format:
 *                 SPLITZIP_FORMAT_BF16, to which every format widens exactly
 *                 (exponent bytes other than those that the store writes: to
 *                 nearest even), or SPLITZIP_FORMAT_E5M2 from a pool of E5M2
 * tokens <= table_width * page_tokens, tokens < 2^31 - 256; 2 * batch * kv_heads *
 * (tokens + 31) / 32 < 2^31.  One launch. */
typedef struct splitzip_pages_load_args {
    splitzip_pool pool;
    const int32_t *table, *lens;
    splitzip_view k_out, v_out;
    uint32_t batch, tokens, table_width, out_format;
} splitzip_pages_load_args;

splitzip_status splitzip_pages_load(const splitzip_pages_load_args *args, splitzip_stream_t s);

/* -------------------------------------------------------------- attention */

/* Attention of the new tokens of a batch, packed one after the other: sequence
 * b's are rows q_start[b] .. q_start[b + 1] - 1 of q, its last tokens.  With n =
 * lens[b] (clamped to [0, kv_tokens]) and m new tokens, new token i is at position
 * p = n - m + i and sees token t if t <= p and (window = 0 or t > p - window or
 * t < sinks); at a negative position it sees nothing.  Query head h reads
 * key/value head h / (q_heads / kv_heads).
 *   q, out   BF16 [tokens, q_heads, head_dim]; rows of out (and lse) that are no
 *            sequence's, such as padding behind the last one, stay as they were
 *   lse      float[q_heads][tokens], may be NULL
 *   table    int32[batch][table_width]; entries whose tokens no query sees (behind
 *            a sequence's last one, or left by its window) are not looked at; where
 *            a query sees a token whose page is outside the pool, its out and lse,
 *            and those of queries near it, are NaN
 *   q_start  int32[batch + 1]; a sequence whose range does not lie in [0, tokens]
 *            or holds more than max_q_tokens is left out; where starts that go back
 *            make ranges overlap, out and lse are unspecified
 *   lens     int32[batch], with the new tokens counted
 * Scores, the softmax statistics and sums are held in 32 bits.  A weight enters its
 * product with the values in 16 bits, and so counts for out, but not for lse: BF16
 * over BF16 pages (off by up to 2^-8 of itself), FP16 over all others (2^-11, below
 * 2^-22 of the row's largest by up to 2^-33 of that).  Over those a query too is
 * FP16, of its row scaled by a power of two: values down to 2^-17 of the row's
 * largest keep all their bits.  A query that sees nothing, or scores of -infinity
 * alone, gets out = 0 and lse = -inf.  Tokens
 * that a query does not see contribute nothing to it, whatever their slots hold;
 * where it sees a quantised token whose exponent bytes are not ones that the store
 * writes, its out and lse are unspecified.
 * q_heads a multiple of kv_heads, at most SPLITZIP_MAX_GROUP times it; scale
 * positive and finite; kv_tokens <= table_width * page_tokens; max_q_tokens <=
 * tokens; tokens * (q_heads / kv_heads) and kv_tokens at most 2^31 - 256; batch *
 * kv_heads * tokens < 2^31. */
typedef struct splitzip_paged_attention_args {
    splitzip_view q, out;
    splitzip_pool pool;
    float *lse;
    const int32_t *table, *q_start, *lens;
    uint32_t batch, tokens, max_q_tokens, kv_tokens, table_width, q_heads;
    uint32_t window, sinks;
    float scale;
} splitzip_paged_attention_args;

/* Bytes of workspace for these sizes (pointers, strides and scale are not looked
 * at), as splitzip_attention_workspace_bytes: zero-filled once, shared by calls
 * that are ordered on one stream and need no more than it holds, also with those
 * of splitzip_attention.  Smaller sizes may need more: fewer sequences are split
 * into more parts.  0 for sizes that are refused.
 *
 * Over pages other than BF16 a sequence of more than 1024 query rows (new tokens
 * times the heads of a group; 2048 in E5M2 at head_dim 128) has its cache widened
 * to 16 bits in the workspace first, so there is room for as many sequences as may
 * have more: each 4 bytes a value of kv_tokens (rounded up to 128) * kv_heads *
 * head_dim.  If that is above 4 GiB none is, and the pages are widened again for
 * every 256 rows, which takes longer (2048 tokens of 32 heads over 8k tokens of 8
 * heads of 128 in 8 bits: 215 us in place of 188).  It goes by max_q_tokens for a
 * batch of one: a token under a bound of 2048 has its whole cache widened. */
size_t splitzip_paged_attention_workspace_bytes(const splitzip_paged_attention_args *args);

/* splitzip_attention_status reports on the workspace. */
splitzip_status splitzip_paged_attention(const splitzip_paged_attention_args *args, void *workspace,
                                         size_t workspace_bytes, splitzip_stream_t s);

#ifdef __cplusplus
}
#endif

#endif /* SPLITZIP_PAGES_H */
