// Where kernels record what they find wrong with a call's inputs (codes from
// 0x201 on).  It is a word beside g_device_error, which the waits that ran out
// own: running out of pages is an ordinary event of a server, and must not hide
// a wait that runs out before somebody has read it.
#pragma once
#include "common.cuh"

namespace sa {

__device__ int g_input_error;

// The first one stays.
__device__ __forceinline__ void report_input(int code) { atomicCAS(&g_input_error, 0, code); }

}  // namespace sa
