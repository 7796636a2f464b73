// early.cuh -- kernels that are launched while the one before them on the stream still
// ends, so that its last CTAs and the launch itself overlap (2 us a call in a stream of
// calls: 8192 x 20 head rows 20.0 -> 17.4 us).
//
// Such a kernel's first act, by every thread, is wait_earlier(): behind it everything that
// came before on the stream is complete and can be seen.  It has to be every thread's, as a
// kernel launched behind this one waits for this one's end alone.  Tensors are read by
// plain loads, or past L1, and not as data that is read-only for the kernel's life (which
// begins before the wait).
#pragma once

#include <cuda_runtime.h>

#include "internal.h"

namespace moe {

__device__ __forceinline__ void wait_earlier() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
int launch_early(void (*kern)(P...), int64_t grid, int threads, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...) == cudaSuccess ? MOE_OK : MOE_ECUDA;
}

}  // namespace moe
