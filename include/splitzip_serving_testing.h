/*
 * splitzip_serving_testing.h -- test controls of the operators around the KV cache
 * (not for production callers).
 *
 * The attention of many query rows and the attention weight are computed by
 * kernels whose warps hand tiles to one another.  Every wait for a tile is
 * bounded; when one runs out the CTA's other waits end too, its results are NaN,
 * the copies in flight are waited for, its tensor memory is given back and the
 * kernel returns, leaving the CUDA context usable.  These entry points let a test
 * make a wait run out on purpose: a copy of one tile is left out, so that what
 * waits for it gives up after a short limit.  Nothing faults or hangs.
 */
#ifndef SPLITZIP_SERVING_TESTING_H
#define SPLITZIP_SERVING_TESTING_H

#include "splitzip_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct splitzip_wait_test_opts {
    uint32_t wait_ms; /* what a wait may last, at most 2000; 0: the default */
    uint32_t cta;     /* the CTA, and which of the tiles that it copies (keys and values in */
    uint32_t tile;    /* turn; keys and queries for the weights) is left out; none past the end */
} splitzip_wait_test_opts;

/* splitzip_attention with test controls.  Sizes whose kernel has no such waits
 * (few query rows) are refused. */
splitzip_status splitzip_attention_test(const splitzip_attention_args *args, void *workspace,
                                        size_t workspace_bytes, splitzip_stream_t s,
                                        const splitzip_wait_test_opts *opts);

/* splitzip_attention_weights with test controls. */
splitzip_status splitzip_attention_weights_test(const splitzip_attention_args *args,
                                                const float *weights_in, float *weights_out,
                                                splitzip_stream_t s,
                                                const splitzip_wait_test_opts *opts);

#ifdef __cplusplus
}
#endif

#endif /* SPLITZIP_SERVING_TESTING_H */
