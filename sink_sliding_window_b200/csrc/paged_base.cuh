// What all kernels of the paged cache share.  (Not in common.cuh and ptx.cuh:
// those are part of the backward's kernel, whose committed profile is of
// exactly its sources.)
#pragma once
#include "common.cuh"
#include "input_error.cuh"

namespace sa {

// Codes of what only the device can see of a call's inputs (see DeviceError).
enum PagedError : int {
  kDevErrPoolExhausted = 0x202,  // a planned step wanted more pages than the pool holds
  kDevErrBadPage = 0x203,        // a needed block-table entry, pool entry or slot lies outside the pool
  kDevErrPlanLengths = 0x204,    // a request's lengths do not fit its table row, or the step its slot map
  kDevErrPagedRows = 0x205,      // cu_seqlens do not fit total_tokens, or a request has more than max_new tokens
};

// Programmatic dependent launch.  A kernel launched so may start while the one
// before it on the stream runs, as soon as all CTAs of that one have allowed it
// (launch_dependents) or ended; pdl_wait() returns when that one and all before
// it have ended and what they wrote can be read.  Without such a launch both do
// nothing.
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Orders this thread's generic-proxy view of global memory before its later TMA
// copies from there.
__device__ __forceinline__ void fence_proxy_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}

}  // namespace sa
