// launch_after.cuh -- a kernel that follows another of the same call: its launch and the start of its CTAs overlap
// the other's work (programmatic dependent launch).
#pragma once

#include <utility>

#include <cuda_runtime.h>

namespace kda {

// In the kernel before (never a call's last one): from here on, once all of its CTAs have come here, the next
// one's may be placed.  A kernel that takes TMEM calls it behind the barrier that follows its allocation: a CTA of
// the next one on the same SM could otherwise take the columns first and wait for this kernel, which waits for them
// (an allocation has no limit); only the two kernels' registers and shared memory would keep that from happening.
// For kernels whose CTAs fill the machine once (linear attention of 2 x 2048 tokens, 16
// heads of 128: 38.5 -> 35.8 us, its gradients 100.7 -> 97.7, the norms' 2 us less).  Before kernels of many small
// CTAs it loses, since those are then placed unevenly (gradients of 8192 tokens: token walks, 4 heads of 64, fp32,
// 445 -> 499 us; chains, 16 heads of 64, 117 -> 146 us): the kernels before them leave it to their end.
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// In the kernel after: every kernel before it in the call has ended and its writes are visible.  At least one
// thread of the grid has to come here even where it reads nothing of theirs, since what follows the call in the
// stream waits for the last kernel alone.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A &&...args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace kda
