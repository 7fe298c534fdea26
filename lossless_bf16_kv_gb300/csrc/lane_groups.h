// lane_groups.h -- which item of work a thread's group of lanes takes (host and
// device; plain C++, so that the host can check it).
#pragma once

#include <cstdint>

namespace splitzip {

// The number, over the grid, of the group of `lanes` threads that thread `thread`
// of CTA `block` belongs to; `threads` per CTA, a multiple of `lanes`.  The grid may
// hold more than 2^32 threads, but not that many groups: no product here counts threads.
#ifdef __CUDACC__
__host__ __device__ __forceinline__
#else
inline
#endif
    uint32_t
    lane_group(uint32_t block, uint32_t thread, uint32_t threads, uint32_t lanes) {
    return block * (threads / lanes) + thread / lanes;
}

}  // namespace splitzip
