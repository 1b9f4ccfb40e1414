// Device helpers of the 8-bit integer products.
#pragma once

#include <type_traits>

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

// silu(g) * u to a few ulps of fp32 (g > -87; below, exp(-|g|) is subnormal):
// the exponential within an ulp, and neither it nor the quotient overflows.  (The
// hardware's exponential rounds its argument first and is off by |g| 2^-24.)
__device__ __forceinline__ float silu_mul(float g, float u) {
    const float e = expf(-fabsf(g));
    return (g < 0.f ? e == 0.f ? 0.f : g * e : g) / (1.f + e) * u;
}

// A scale as mant * 2^exp, |mant| in [1/2, 1): the product of a row's and a
// channel's scale may leave fp32's normal range where the result does not.
struct Scale {
    float mant;
    int exp;
};
__device__ __forceinline__ Scale split(float s) {
    return Scale{__builtin_amdgcn_frexp_mantf(s), __builtin_amdgcn_frexp_expf(s)};
}
// a * b * sum.  The powers of two are exact: the bits are those of the three
// factors' product in fp32 wherever that stays in range.
__device__ __forceinline__ float scaled(Scale a, Scale b, int32_t sum) {
    return __builtin_ldexpf(a.mant * b.mant * (float)sum, a.exp + b.exp);
}

// y as T.  An fp16 is rounded from the fp32 value like everywhere else: folded
// into one instruction with the sum that makes y, it would be rounded once where
// the other kernels round twice, and a row's bits would follow the kernel.
template <typename T>
__device__ __forceinline__ T as_type(float y) {
    if constexpr (std::is_same_v<T, _Float16>) asm("" : "+v"(y));
    return (T)y;
}

// Offsets of experts e0 + 64 c + lane, c < 4, all loads in flight together.
struct Offsets4 {
    int o0[4], o1[4];
};
__device__ __forceinline__ Offsets4 load_offsets(const int32_t* offsets, int E, int e0, int lane) {
    Offsets4 o;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int e = e0 + 64 * c + lane;
        o.o0[c] = e < E ? offsets[e] : 0;
        o.o1[c] = e < E ? offsets[e + 1] : 0;
    }
    return o;
}

}  // namespace moeq
