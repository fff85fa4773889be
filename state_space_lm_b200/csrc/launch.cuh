// launch.cuh -- launches of several kernels in a row (not part of the ABI).
//
// Short kernels of one call that follow another of its kernels are launched as
// that one's programmatic dependents: their set-up passes while the kernel
// before them drains (group norm over sequences, backward, 8 x 2048 x 1024: 51
// to 47 us).  The passes of the mixes are not: a CTA of theirs holds an SM, and
// one that waits there was slower.  A kernel calls pdl_trigger() at its start,
// and pdl_wait() before it reads what the kernels before it in the call wrote
// (it returns when those have finished, with their memory visible).  The call's
// first kernel is launched as usual, after everything earlier on the stream; so
// the call's own inputs may be read before pdl_wait().  Every block of a
// dependent waits before it ends: then a kernel that has finished says that all
// before it have.
#pragma once
#include "m3_internal.cuh"

namespace m3 {

__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, A &&...args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&c, kernel, P(args)...);
    if (e == cudaSuccess) count_launch();
    return e;
}

}  // namespace m3
