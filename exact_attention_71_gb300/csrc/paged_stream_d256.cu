// Paged attention, streaming kernel at head_dim 256.
#include "paged_stream_launch.cuh"

namespace attn {

cudaError_t run_paged_stream_d256(const PagedParams& p, bool prefix, bool direct, cudaStream_t stream) {
    return launch_paged_stream<256>(p, prefix, direct, stream);
}

}  // namespace attn
