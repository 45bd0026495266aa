// Host-side launch of the tile kernel's instantiations.
#pragma once

#include "paged_tile_kernel.cuh"

namespace attn {

template <class Cfg, bool DIRECT, bool TREE>
cudaError_t launch_paged_tile_one(const PagedMaps& m, const PagedParams& p, cudaStream_t stream) {
    auto kernel = paged_tile_kernel<Cfg, DIRECT, TREE>;
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = once_per_device(ready, [&] {
        // The register split (setmaxnreg) assumes exactly LAUNCH_REGS registers
        // a thread at launch; another count could make the increase wait
        // forever, so such a build is refused.
        cudaFuncAttributes attr;
        cudaError_t r = cudaFuncGetAttributes(&attr, kernel);
        if (r != cudaSuccess) return r;
        if (attr.numRegs != Cfg::LAUNCH_REGS) return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
    });
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, p.prefix_items + p.own_items, Cfg::THREADS, Cfg::SMEM_BYTES, false, stream, m.k, m.v, p);
}

template <int D, bool TREE>
cudaError_t launch_paged_tile(const PagedMaps& m, const PagedParams& p, bool direct, cudaStream_t stream) {
    if (p.fp8) {
        using C = TileCfg<D, true>;
        return direct ? launch_paged_tile_one<C, true, TREE>(m, p, stream) : launch_paged_tile_one<C, false, TREE>(m, p, stream);
    }
    using C = TileCfg<D, false>;
    return direct ? launch_paged_tile_one<C, true, TREE>(m, p, stream) : launch_paged_tile_one<C, false, TREE>(m, p, stream);
}

}  // namespace attn
