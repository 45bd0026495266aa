// Paged attention, tile kernel at head_dim 64.
#include "paged_tile_launch.cuh"

namespace attn {

cudaError_t run_paged_tile_d64(const PagedMaps& m, const PagedParams& p, bool direct, cudaStream_t stream) {
    return launch_paged_tile<64>(m, p, direct, stream);
}

}  // namespace attn
