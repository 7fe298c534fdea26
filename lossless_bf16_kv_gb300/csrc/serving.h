// serving.h -- launch arguments and launchers of the operators around the KV
// cache (internal; the public interface is include/splitzip_serving.h).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/splitzip_serving.h"

namespace splitzip {

cudaError_t launch_norm_rope(const splitzip_norm_rope_args& a, cudaStream_t s);

// How a call's query rows (query token, query head of one key/value head) are
// cut into row tiles and each tile's slots into splits.
// The workspace starts with a header that has the same place whatever the
// sizes: a counter per row tile that has splits (at most kSms; zero between
// calls) and the status bits that a call leaves.  The splits' partial results
// follow.
constexpr size_t kAttentionHeader = 1024, kAttentionStatus = 1020;
struct AttentionPlan {
    uint32_t rows;       // q_tokens * group, of one key/value head
    uint32_t row_tiles;  // of tile_rows rows
    uint32_t tile_rows;
    uint32_t splits;     // parts of one row tile's slots, joined at the end
    size_t bytes;        // of workspace
};
// Few query rows (attention_rows.cu) and many (attention_tiles.cu).  A plan
// depends on the sizes alone; it is false where they do not fit a launch.
bool attention_rows_plan(const splitzip_attention_args& a, AttentionPlan& p);
bool attention_tiles_plan(const splitzip_attention_args& a, AttentionPlan& p);
bool attention_tiles_usable(const splitzip_attention_args& a);
cudaError_t launch_attention_rows(const splitzip_attention_args& a, const AttentionPlan& p,
                                  void* workspace, cudaStream_t s);
// A CTA whose tile-th copy is left out, and the limit of the waits (0: as it is
// otherwise), for tests of what happens then.
struct WaitTest {
    uint32_t limit = 0, cta = 0xFFFFFFFFu, tile = 0xFFFFFFFFu;
};
cudaError_t launch_attention_tiles(const splitzip_attention_args& a, const AttentionPlan& p,
                                   void* workspace, const WaitTest& test, cudaStream_t s);
cudaError_t launch_attention_weights(const splitzip_attention_args& a, const float* weights_in,
                                     float* weights_out, const WaitTest& test, cudaStream_t s);
cudaError_t launch_evict(const splitzip_evict_args& a, cudaStream_t s);

}  // namespace splitzip
