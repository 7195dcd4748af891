// Programmatic dependent launch inside one call: a kernel may start while its
// predecessor on the stream still runs, does what needs none of its results
// (barriers, tensor memory, index arithmetic), and then waits for it to end.
// A call's first kernel is launched plainly, so that calls stay ordered as
// kernels on a stream are; every kernel of a chain waits, so that a kernel's
// end implies the end of all before it.
#pragma once
#include <cuda_runtime.h>

namespace muon {

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

#ifdef __CUDACC__
// The predecessor's kernel has ended and its writes are visible.
__device__ __forceinline__ void wait_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The successor may start (it waits for this kernel's end before it reads).
__device__ __forceinline__ void allow_successor() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

}  // namespace muon
