// paged_tiles_128_twin.cu -- the kernels of paged_tiles.cuh for head_dim 128, twin tiles (sm_103a).
#include "paged_tiles.cuh"

namespace splitzip {

cudaError_t launch_paged_128_twin(const PagedTilesParams& p, uint32_t ctas, bool beside, cudaStream_t s) {
    return launch_paged_format<128, true>(p, ctas, beside, s);
}

}  // namespace splitzip
