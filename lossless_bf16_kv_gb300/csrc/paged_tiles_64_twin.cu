// paged_tiles_64_twin.cu -- the kernels of paged_tiles.cuh for head_dim 64, twin tiles (sm_103a).
#include "paged_tiles.cuh"

namespace splitzip {

cudaError_t launch_paged_64_twin(const PagedTilesParams& p, uint32_t ctas, bool beside, cudaStream_t s) {
    return launch_paged_format<64, true>(p, ctas, beside, s);
}

}  // namespace splitzip
