// pages.h -- launch arguments and launchers of the paged cache's operators
// (internal; the public interface is include/splitzip_pages.h).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/splitzip_pages.h"
#include "serving.h"

namespace splitzip {

cudaError_t launch_pages_store(const splitzip_pages_store_args& a, cudaStream_t s);
cudaError_t launch_pages_load(const splitzip_pages_load_args& a, cudaStream_t s);

// Sequences of few query rows (new tokens times the heads of a group; paged_rows.cu)
// and of many (paged_tiles.cu).  A plan depends on the sizes alone; it is false where
// they do not fit a launch.
struct PagedPlan {
    uint32_t row_tiles;  // of a sequence (few rows), or at most of the batch (many)
    uint32_t splits;     // 0 (few rows): by the sequences' lengths
    uint64_t ctas;       // of the launch
    size_t bytes;        // of workspace: from its start (few rows), or of partial results (many)
};
// Sequences of up to rows_upto query rows, and of more than rows_from, up to rows_upto.
bool paged_rows_plan(const splitzip_paged_attention_args& a, uint32_t rows_upto, PagedPlan& p);
bool paged_tiles_plan(const splitzip_paged_attention_args& a, uint32_t rows_from, uint32_t rows_upto, PagedPlan& p);
// after_tiles: the launch ahead of it is launch_paged_tiles of the same call, whose end it
// need not wait for to start.
cudaError_t launch_paged_rows(const splitzip_paged_attention_args& a, uint32_t rows_upto, const PagedPlan& p, void* workspace,
                              bool after_tiles, const WaitTest& test, cudaStream_t s);
// The bytes of the workspace's header that count the pieces of row tiles, behind those
// that count the splits of few rows.
constexpr size_t kTilesCounters = 640;
// at_partials: where the plan's partial results lie in the workspace, apart from those of
// the call's other launches, which may run at the same time.
// beside: the launch ahead of it is another of the same call, whose end it need not wait
// for.  widened: the sequences' caches in FP16, as launch_paged_widen leaves them (or
// NULL: they are read from the pool).
cudaError_t launch_paged_tiles(const splitzip_paged_attention_args& a, uint32_t rows_from, uint32_t rows_upto, const PagedPlan& p, void* workspace,
                               size_t at_partials, const void* widened, bool beside, const WaitTest& test, cudaStream_t s);

// The caches of a batch's long sequences (more than rows_from query rows) in FP16, one
// after the other in the batch's order: keys, then values, head by head, of
// widened_tokens tokens each.
inline uint64_t widened_sequences(const splitzip_paged_attention_args& a, uint32_t rows_from) {
    const uint64_t rows = (uint64_t)a.tokens * (a.q_heads / a.pool.kv_heads);
    return rows / (rows_from + 1) < a.batch ? rows / (rows_from + 1) : a.batch;
}
inline uint64_t widened_tokens(const splitzip_paged_attention_args& a) { return ((uint64_t)a.kv_tokens + 127) / 128 * 128; }
inline uint64_t widened_bytes(const splitzip_paged_attention_args& a, uint32_t rows_from) {
    return widened_sequences(a, rows_from) * widened_tokens(a) * a.pool.kv_heads * a.pool.head_dim * 4;
}
cudaError_t launch_paged_widen(const splitzip_paged_attention_args& a, uint32_t rows_from, void* widened, cudaStream_t s);

// Whether a page's exponent bytes of a head are contiguous and may be copied in
// multiples of 16 bytes.
inline bool bulk_exponents(const splitzip_pool& p) {
    const auto ok = [&](const splitzip_page_rows& r) {
        return r.exp_stride_t == 4 && (uintptr_t)r.exponents % 16 == 0 && (p.pages == 1 || r.exp_stride_p % 16 == 0) &&
               (p.kv_heads == 1 || r.exp_stride_h % 16 == 0);
    };
    return (p.format == SPLITZIP_FORMAT_INT8 || p.format == SPLITZIP_FORMAT_E2M1) && ok(p.k) && ok(p.v);
}

}  // namespace splitzip
