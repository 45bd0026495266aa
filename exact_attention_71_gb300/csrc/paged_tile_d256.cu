// Paged attention, tile kernel at head_dim 256.
#include "paged_tile_launch.cuh"

namespace attn {

cudaError_t run_paged_tile_d256(const PagedMaps& m, const PagedParams& p, bool direct, cudaStream_t stream) {
    return launch_paged_tile<256, false>(m, p, direct, stream);
}

}  // namespace attn
