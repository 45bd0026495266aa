// Paged attention, tile kernel of trees at head_dim 256.
#include "paged_tile_launch.cuh"

namespace attn {

cudaError_t run_paged_tile_tree_d256(const PagedMaps& m, const PagedParams& p, bool direct, cudaStream_t stream) {
    return launch_paged_tile<256, true>(m, p, direct, stream);
}

}  // namespace attn
