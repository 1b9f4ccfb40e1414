// Device helpers of the 8-bit integer products.
#pragma once

#include "elem_dev.h"

namespace moeq {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// Barrier of a workgroup whose waves only meet in LDS: LDS work is waited for,
// global loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + __expf(-g)) * u; }

}  // namespace moeq
