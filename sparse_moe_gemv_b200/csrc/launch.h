// Launch helpers of the operators around the layer. A failure is the call's own: nothing is left in
// the runtime's last-error state for a later call to find, and none is taken from there.
#pragma once

#include <cuda_runtime.h>

namespace redmoe {

// Allow `kern` (a __global__ function) `bytes` of dynamic shared memory on the current device. What
// has been allowed is remembered, so a call that asks again costs a lookup; false on a CUDA error.
bool allow_smem(const void* kern, int bytes);

// kern(args...) in clusters of `cluster` blocks. The blocks may be placed while the kernel before on the
// stream ends; the kernel waits for that end itself (wait_for_previous).
template <class... P, class... A>
bool launch(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, int cluster, A... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess) return true;
    cudaGetLastError();
    return false;
}

#ifdef __CUDACC__
// In every kernel launched so, before it reads or writes global memory. What kernels before it
// wrote is then visible to plain loads; loads through the read-only path (ld.global.nc) are not used
// in such kernels, since their data would have to stay unchanged from the kernel's start.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// From here on (in all blocks) the next kernel on the stream may take room that is left, to wait there.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }
#endif

}  // namespace redmoe
