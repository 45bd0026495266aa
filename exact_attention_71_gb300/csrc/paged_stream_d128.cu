// Paged attention, streaming kernel at head_dim 128.
#include "paged_stream_launch.cuh"

namespace attn {

cudaError_t run_paged_stream_d128(const PagedMaps& m, const PagedParams& p, bool prefix, bool own, bool direct, bool after,
                                 cudaStream_t stream) {
    return launch_paged_stream<128>(m, p, prefix, own, direct, after, stream);
}

}  // namespace attn
