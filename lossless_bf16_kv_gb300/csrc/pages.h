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

// Sequences by how many query rows (new tokens times heads of a group) they bring.
struct PagedPlan {
    uint32_t row_tiles, splits;
    size_t bytes;  // of workspace
};
bool paged_rows_plan(const splitzip_paged_attention_args& a, PagedPlan& p);
cudaError_t launch_paged_rows(const splitzip_paged_attention_args& a, const PagedPlan& p, void* workspace, cudaStream_t s);

}  // namespace splitzip
