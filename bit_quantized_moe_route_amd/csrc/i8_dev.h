// Device helpers of the 8-bit integer products.
#pragma once

#include "elem_dev.h"

namespace moeq {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// Barrier of a workgroup whose waves only meet in LDS: LDS work is waited for,
// global loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Keeps the order of the program around it: nothing is emitted.
__device__ __forceinline__ void keep_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_sched_barrier(0);
}

// A value that is the same in every lane, in a scalar register: what branches
// around matrix instructions go by, which run whatever the lane mask says.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + __expf(-g)) * u; }

}  // namespace moeq
