// Paged attention, streaming kernel at head_dim 64.
#include "paged_stream_launch.cuh"

namespace attn {

cudaError_t run_paged_stream_d64(const PagedParams& p, bool prefix, bool direct, cudaStream_t stream) {
    return launch_paged_stream<64>(p, prefix, direct, stream);
}

}  // namespace attn
