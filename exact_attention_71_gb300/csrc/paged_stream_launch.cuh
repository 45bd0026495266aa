// Host-side launch of the streaming kernel's instantiations.
#pragma once

#include "paged_stream_kernel.cuh"

namespace attn {

template <class Cfg, bool PREFIX, bool DIRECT>
cudaError_t launch_paged_stream_one(const PagedParams& p, cudaStream_t stream) {
    auto kernel = paged_stream_kernel<Cfg, PREFIX, DIRECT>;
    // Per function and per device; cheap and idempotent.
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const unsigned tiles = ((PREFIX ? p.B : 1) * p.Nq * p.G + 15) / 16;
    const dim3 grid(tiles * p.H_kv * (PREFIX ? p.prefix_parts : p.own_parts), PREFIX ? 1 : p.B);
    kernel<<<grid, Cfg::THREADS, Cfg::SMEM_BYTES, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_paged_stream(const PagedParams& p, bool prefix, bool direct, cudaStream_t stream) {
    if (p.fp8) {
        using C = StreamCfg<D, true>;
        if (prefix) return launch_paged_stream_one<C, true, false>(p, stream);
        return direct ? launch_paged_stream_one<C, false, true>(p, stream)
                      : launch_paged_stream_one<C, false, false>(p, stream);
    }
    using C = StreamCfg<D, false>;
    if (prefix) return launch_paged_stream_one<C, true, false>(p, stream);
    return direct ? launch_paged_stream_one<C, false, true>(p, stream)
                  : launch_paged_stream_one<C, false, false>(p, stream);
}

}  // namespace attn
