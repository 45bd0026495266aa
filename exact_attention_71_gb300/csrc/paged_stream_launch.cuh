// Host-side launch of the streaming kernel's instantiations.
#pragma once

#include "paged_stream_kernel.cuh"

namespace attn {

template <class Cfg, bool DIRECT, bool TREE>
cudaError_t launch_paged_stream_one(const PagedMaps& m, const PagedParams& p, bool prefix, bool own, bool after,
                                    cudaStream_t stream) {
    auto kernel = paged_stream_kernel<Cfg, DIRECT, TREE>;
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = once_per_device(ready, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
    });
    if (e != cudaSuccess) return e;
    const unsigned per = p.Nq * p.G;
    const unsigned prefix_blocks = prefix ? (p.B * per + Cfg::ROWS - 1) / Cfg::ROWS * p.H_kv * p.prefix_parts : 0;
    const unsigned own_blocks = own ? (per + Cfg::ROWS - 1) / Cfg::ROWS * p.H_kv * p.own_parts * p.B : 0;
    return launch_kernel(kernel, prefix_blocks + own_blocks, Cfg::THREADS, Cfg::SMEM_BYTES, after, stream, m.k, m.v, p,
                         prefix_blocks);
}

template <int D, bool FP8, bool TREE>
cudaError_t launch_paged_stream_rows(const PagedMaps& m, const PagedParams& p, bool prefix, bool own, bool direct,
                                     bool after, cudaStream_t stream) {
    if (p.stream_tile == 8)
        return direct ? launch_paged_stream_one<StreamCfg<D, FP8, 1>, true, TREE>(m, p, prefix, own, after, stream)
                      : launch_paged_stream_one<StreamCfg<D, FP8, 1>, false, TREE>(m, p, prefix, own, after, stream);
    return direct ? launch_paged_stream_one<StreamCfg<D, FP8, 2>, true, TREE>(m, p, prefix, own, after, stream)
                  : launch_paged_stream_one<StreamCfg<D, FP8, 2>, false, TREE>(m, p, prefix, own, after, stream);
}

template <int D, bool TREE>
cudaError_t launch_paged_stream(const PagedMaps& m, const PagedParams& p, bool prefix, bool own, bool direct,
                                bool after, cudaStream_t stream) {
    return p.fp8 ? launch_paged_stream_rows<D, true, TREE>(m, p, prefix, own, direct, after, stream)
                 : launch_paged_stream_rows<D, false, TREE>(m, p, prefix, own, direct, after, stream);
}

}  // namespace attn
