// Paged attention, tile kernel at head_dim 128.
#include "paged_tile_launch.cuh"

namespace attn {

cudaError_t run_paged_tile_d128(const PagedParams& p, bool direct, cudaStream_t stream) {
    return launch_paged_tile<128>(p, direct, stream);
}

}  // namespace attn
