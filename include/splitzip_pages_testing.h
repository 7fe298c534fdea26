/*
 * splitzip_pages_testing.h -- test controls of the paged cache's attention (not for
 * production callers), as splitzip_serving_testing.h has them for the strided one's.
 */
#ifndef SPLITZIP_PAGES_TESTING_H
#define SPLITZIP_PAGES_TESTING_H

#include "splitzip_pages.h"
#include "splitzip_serving_testing.h"

#ifdef __cplusplus
extern "C" {
#endif

/* splitzip_paged_attention with test controls.  opts->cta is a CTA of each of the
 * call's attention kernels; opts->tile counts the parts of tiles that it loads (for
 * many query rows keys' and values' in turn, for few both of a tile as one). */
splitzip_status splitzip_paged_attention_test(const splitzip_paged_attention_args *args, void *workspace,
                                              size_t workspace_bytes, splitzip_stream_t s,
                                              const splitzip_wait_test_opts *opts);

#ifdef __cplusplus
}
#endif

#endif /* SPLITZIP_PAGES_TESTING_H */
