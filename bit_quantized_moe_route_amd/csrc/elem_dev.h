// Device-side helpers of the calls that take rows of fp32, bf16 or fp16
// (block norms, 8-bit quantisation): 8-element raw loads, their conversion to
// fp32, rounding stores, and reductions over a workgroup.  gfx950 only.
#pragma once

#include <type_traits>

#include "dev_common.h"

namespace moeq {

// Eight elements as loaded: 16 bytes of a 16-bit type (in a), or 32 of fp32.
// The type is the same for a whole launch, so its branches are uniform; the
// raw words stay unconverted until they are used, so that loads of several
// operands are in flight together.
struct Raw8 {
    u32x4 a, b;
};

// 16 bytes at an element's own alignment (ANY), which the memory path takes as
// they are, or at 16; STREAM: past the caches.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

template <bool STREAM = false, bool ANY = false>
__device__ __forceinline__ u32x4 load16(const void* p) {
    using Q = std::conditional_t<ANY, u32x4_any, u32x4>;
    const Q* q = static_cast<const Q*>(p);
    if constexpr (STREAM) return __builtin_nontemporal_load(q);
    return *q;
}

template <bool STREAM = false, bool ANY = false>
__device__ __forceinline__ void store16(void* p, u32x4 u) {
    using Q = std::conditional_t<ANY, u32x4_any, u32x4>;
    Q* q = static_cast<Q*>(p);
    if constexpr (STREAM) __builtin_nontemporal_store((Q)u, q);
    else *q = u;
}

template <bool STREAM = false, bool ANY = false>
__device__ __forceinline__ Raw8 load_raw8(const void* p, int dt, int64_t i) {
    Raw8 r;
    if (dt == MOE_DT_F32) {
        const float* q = static_cast<const float*>(p) + i;
        r.a = load16<STREAM, ANY>(q);
        r.b = load16<STREAM, ANY>(q + 4);
    } else {
        r.a = load16<STREAM, ANY>(static_cast<const uint16_t*>(p) + i);
        r.b = u32x4{0u, 0u, 0u, 0u};
    }
    return r;
}

__device__ __forceinline__ void raw_to_f32(const Raw8& r, int dt, float (&v)[8]) {
    if (dt == MOE_DT_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(r.a[i]);
            v[4 + i] = __uint_as_float(r.b[i]);
        }
    } else if (dt == MOE_DT_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r.a[i] << 16);
            v[2 * i + 1] = __uint_as_float(r.a[i] & 0xffff0000u);
        }
    } else {
        const f16x8 h = __builtin_bit_cast(f16x8, r.a);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
    }
}

__device__ __forceinline__ float load_elem(const void* p, int dt, int64_t i) {
    if (dt == MOE_DT_F32) return static_cast<const float*>(p)[i];
    const uint16_t u = static_cast<const uint16_t*>(p)[i];
    if (dt == MOE_DT_BF16) return __uint_as_float((uint32_t)u << 16);
    return (float)__builtin_bit_cast(_Float16, u);
}

// V elements (8: one vector, 1: a scalar) as loaded, and as fp32.
template <int V>
struct Raw;
template <>
struct Raw<8> {
    Raw8 r;
    template <bool STREAM = false, bool ANY = false>
    __device__ __forceinline__ void load(const void* p, int dt, int64_t i) {
        r = load_raw8<STREAM, ANY>(p, dt, i);
    }
    __device__ __forceinline__ void f32(int dt, float (&v)[8]) const { raw_to_f32(r, dt, v); }
};
template <>
struct Raw<1> {
    uint32_t r;
    template <bool STREAM = false, bool ANY = false>
    __device__ __forceinline__ void load(const void* p, int dt, int64_t i) {
        r = dt == MOE_DT_F32 ? static_cast<const uint32_t*>(p)[i]
                             : static_cast<const uint16_t*>(p)[i];
    }
    __device__ __forceinline__ void f32(int dt, float (&v)[1]) const {
        v[0] = dt == MOE_DT_F32    ? __uint_as_float(r)
               : dt == MOE_DT_BF16 ? __uint_as_float(r << 16)
                                   : (float)__builtin_bit_cast(_Float16, (uint16_t)r);
    }
};

template <int V, bool ANY = false>
__device__ __forceinline__ void load_f32(const void* p, int dt, int64_t i, float (&v)[V]) {
    if constexpr (V == 8) {
        raw_to_f32(load_raw8<false, ANY>(p, dt, i), dt, v);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = load_elem(p, dt, i + e);
    }
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// fp32 -> bf16 bits of a pair, nearest even (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)lo, (_Float16)hi});
}

// One rounding to the stored type, nearest even.  STREAM: results that no
// cache will hold until they are read (8 elements at a time only).
template <int V, bool STREAM = false, bool ANY = false>
__device__ __forceinline__ void store_f32(void* p, int dt, int64_t i, const float (&v)[V]) {
    if constexpr (V == 8) {
        u32x4 u;
        if (dt == MOE_DT_F32) {
            float* q = static_cast<float*>(p) + i;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int e = 0; e < 4; ++e) u[e] = __float_as_uint(v[4 * h + e]);
                store16<STREAM, ANY>(q + 4 * h, u);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                u[e] = dt == MOE_DT_BF16 ? pack_bf16(v[2 * e], v[2 * e + 1])
                                         : pack_f16(v[2 * e], v[2 * e + 1]);
            store16<STREAM, ANY>(static_cast<uint16_t*>(p) + i, u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (dt == MOE_DT_F32)
                static_cast<float*>(p)[i + e] = v[e];
            else
                static_cast<uint16_t*>(p)[i + e] =
                    (uint16_t)(dt == MOE_DT_BF16 ? pack_bf16(v[e], 0.f) : pack_f16(v[e], 0.f));
        }
    }
}

// Elements lo .. V - 1 of a chunk (lo <= 0: all of it, at i and on).
template <int V, bool STREAM, bool ANY>
__device__ __forceinline__ void store_from(void* p, int dt, int64_t i, const float (&v)[V],
                                           int lo) {
    if (!ANY || lo <= 0) {
        store_f32<V, STREAM, ANY>(p, dt, i, v);
    } else {
#pragma unroll
        for (int e = 1; e < V; ++e) {
            const float one[1] = {v[e]};
            if (e >= lo) store_f32<1>(p, dt, i + e, one);
        }
    }
}

// Four neighbours, aligned to four elements.
__device__ __forceinline__ void store_quad(void* p, int dt, int64_t i, const float (&v)[4]) {
    if (dt == MOE_DT_F32) {
        *reinterpret_cast<f32x4*>(static_cast<float*>(p) + i) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
        const bool b = dt == MOE_DT_BF16;
        const uint2 u = {b ? pack_bf16(v[0], v[1]) : pack_f16(v[0], v[1]),
                         b ? pack_bf16(v[2], v[3]) : pack_f16(v[2], v[3])};
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = u;
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
    return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off));
    return v;
}

// Over the workgroup's nw waves, in wave order (the same bits in every
// thread); red: one word per wave, not in use by another reduction.
__device__ __forceinline__ float block_sum(float v, float* red, int nw) {
    v = wave_sum(v);
    if (nw == 1) return v;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < nw; ++i) t += red[i];
    return t;
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red, int nw) {
    v = wave_max(v);
    if (nw == 1) return v;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    uint32_t t = 0u;
    for (int i = 0; i < nw; ++i) t = max(t, red[i]);
    return t;
}

// The 8-bit code of a row: its scale and multiplier from the largest |v| of
// the row (its bits: as integers they order like the magnitudes, and a NaN
// or an infinity comes out above every finite value).
//   finite a >= 127 * 2^-126:  scale a / 127, codes rint(127 v / a)
//   smaller a (a row of zeros): scale 0, codes 0
//   a row with an infinity or a NaN: scale NaN, codes 0
struct RowCode {
    float scale;
    double mul;
};
__device__ __forceinline__ RowCode row_code(uint32_t amax_bits) {
    const float a = __uint_as_float(amax_bits);
    if (amax_bits >= 0x7f800000u) return RowCode{__uint_as_float(0x7fc00000u), 0.};
    if (a < 127.f * 0x1p-126f) return RowCode{0.f, 0.};
    // 127 / a to fp64's precision: the instruction's 2^-24 squared, and again.  (A
    // full fp64 division in every wave: 4096 x 6145 bf16 26.4 us against 24.8.)
    const double d = a;
    double y = __builtin_amdgcn_rcp(d);
    y = __builtin_fma(__builtin_fma(-d, y, 1.), y, y);
    const double m = 127. * y;
    return RowCode{a / 127.f, __builtin_fma(__builtin_fma(-d, m, 127.), y, m)};
}

// rint(127 v / a), ties to even, in the low byte (mul = 127 / a, not 0).
//   A tie needs more than fp32: |v| = a / 2 is common in 16-bit rows, and v times
// a rounded 127 / a can lie on either side of 63.5.  In fp64 the product is
// within 2^-45 of the quotient.  For fp32 v and a with |127 v / a| > 0.49 a
// quotient that is no tie is at least 2^-33 away from one (v = V 2^-s in units
// of a = A's last place, V and A integers below 2^24 and s <= 8: the distance is
// a whole number of 1 / (2^(s + 1) A)).  So the quotient is first rounded to
// multiples of 2^-36 (the first sum), which puts a tie on itself and moves
// nothing else onto one, and then to integers (the second), where the low byte
// of the mantissa is the code.  Three fp64 instructions: 4096 x 6144 bf16 in
// 22.2 us, 21.3 with one fp32 product.
__device__ __forceinline__ uint32_t code_of(float v, double mul) {
    const double grid = __builtin_fma((double)v, mul, 0x1.8p16);
    return (uint32_t)__double_as_longlong(grid + (0x1.8p52 - 0x1.8p16)) & 0xffu;
}
// Four codes; mul 0 gives 0 whatever v is.
__device__ __forceinline__ uint32_t pack_codes4(const float* v, double mul) {
    uint32_t u = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) u |= code_of(v[e], mul) << (8 * e);
    return mul == 0. ? 0u : u;
}
__device__ __forceinline__ int8_t code1(float v, double mul) {
    return mul == 0. ? (int8_t)0 : (int8_t)code_of(v, mul);
}

}  // namespace moeq
