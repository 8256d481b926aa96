// Launch of a kernel as a programmatic dependent of the one before it in the
// stream (each of the paged-cache kernels waits for that grid before it touches
// global memory); an ordinary launch where that is not available.
#pragma once

#include <cuda_runtime.h>

#include "internal.h"

namespace eta {

template <typename... P, typename... A>
int launch_dependent(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...) == cudaSuccess) return kOk;
    (void)cudaGetLastError();
    cfg.numAttrs = 0;
    if (cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...) == cudaSuccess) return kOk;
    (void)cudaGetLastError();
    return kErrCuda;
}

}  // namespace eta
