// pa_prefill_launch.cuh -- instantiates the chunk attention kernel for one operand family
// and dispatches on head size and block size; each pa_prefill_*.cu includes it once, so
// that the families compile in parallel.
#pragma once

#include "pa_prefill.cuh"

namespace pa {

template <class C>
cudaError_t launch_prefill_one(const CUtensorMap& qmap, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, const PrefillParams& p,
                               cudaStream_t stream) {
    constexpr size_t smem = pf::smem_bytes<C>();
    static_assert(smem <= 227 * 1024, "shared memory");
    auto kern = pf::prefill_kernel<C>;
    static PerDeviceOnce configured;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = static_cast<cudaError_t>(configured.run(dev, [&] {
        // the register split among the warpgroups is written for this count per thread; an
        // increase that the decreases do not cover would wait forever
        cudaFuncAttributes fa;
        cudaError_t e1 = cudaFuncGetAttributes(&fa, kern);
        if (e1 != cudaSuccess) return e1;
        if (fa.numRegs != pf::kRegLaunch) return cudaErrorInvalidKernelImage;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    }));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.grid);
    cfg.blockDim = dim3(pf::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, qmap, kmap, vmap, p);
}

}  // namespace pa
