// dependent.cuh -- device helpers of the kernels launched by launch_dependent, and the untiled
// bulk copy.
#pragma once

#include "mxq_device.cuh"

namespace mxq {

// ---- programmatic dependent launch ---------------------------------------------------

// Wait until the kernel before this one in the stream has ended and its writes are visible
// (returns at once where the launch made no such dependence).  Every kernel launched by
// launch_dependent does this, in every thread, before any access to global memory.
__device__ __forceinline__ void grid_depend_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Let the next kernel's CTAs become resident as this one's leave room (they wait in their own
// grid_depend_wait).
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void grid_wait() {
    grid_depend_wait();
    grid_release();
}

// ---- bulk copy --------------------------------------------------------------------------

// Untiled bulk copy from global to shared memory, completing on `bar`: both addresses
// 16-byte aligned, `bytes` a multiple of 16.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

}  // namespace mxq
