// Host-side launch of the streaming kernel's instantiations.
#pragma once

#include "paged_stream_kernel.cuh"

namespace attn {

template <class Cfg, bool DIRECT>
cudaError_t launch_paged_stream_one(const PagedMaps& m, const PagedParams& p, bool prefix, bool own, bool after,
                                    cudaStream_t stream) {
    auto kernel = paged_stream_kernel<Cfg, DIRECT>;
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = once_per_device(ready, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
    });
    if (e != cudaSuccess) return e;
    const unsigned per = p.Nq * p.G;
    const unsigned prefix_blocks = prefix ? (p.B * per + 15) / 16 * p.H_kv * p.prefix_parts : 0;
    const unsigned own_blocks = own ? (per + 15) / 16 * p.H_kv * p.own_parts * p.B : 0;
    return launch_kernel(kernel, prefix_blocks + own_blocks, Cfg::THREADS, Cfg::SMEM_BYTES, after, stream, m.k, m.v, p,
                         prefix_blocks);
}

template <int D>
cudaError_t launch_paged_stream(const PagedMaps& m, const PagedParams& p, bool prefix, bool own, bool direct,
                                bool after, cudaStream_t stream) {
    if (p.fp8) {
        using C = StreamCfg<D, true>;
        return direct ? launch_paged_stream_one<C, true>(m, p, prefix, own, after, stream)
                      : launch_paged_stream_one<C, false>(m, p, prefix, own, after, stream);
    }
    using C = StreamCfg<D, false>;
    return direct ? launch_paged_stream_one<C, true>(m, p, prefix, own, after, stream)
                  : launch_paged_stream_one<C, false>(m, p, prefix, own, after, stream);
}

}  // namespace attn
