// Paged attention, streaming kernel at head_dim 64.
#include "paged_stream_launch.cuh"

namespace attn {

cudaError_t run_paged_stream_d64(const PagedMaps& m, const PagedParams& p, bool prefix, bool own, bool direct, bool after,
                                 cudaStream_t stream) {
    return launch_paged_stream<64>(m, p, prefix, own, direct, after, stream);
}

}  // namespace attn
