// Paged attention, tile kernel of trees at head_dim 64.
#include "paged_tile_launch.cuh"

namespace attn {

cudaError_t run_paged_tile_tree_d64(const PagedMaps& m, const PagedParams& p, bool direct, cudaStream_t stream) {
    return launch_paged_tile<64, true>(m, p, direct, stream);
}

}  // namespace attn
