// The norm of each query and key head and its rotation by the token's position,
// in one pass.  Per token t and head h, v its D elements, in fp32:
//
//   n = w ? v / sqrt(mean(v^2) + eps) * (w_offset + w) : v
//   for the pairs (a, b) of n's first R elements, (cos, sin) of pair i at pos[t]:
//   a' = a cos - b sin,  b' = b cos + a sin          (pair i: elements i and R/2 + i,
//                                                     or 2i and 2i + 1)
//
// A lane owns units of 2 V elements that hold whole pairs: V neighbours and their V
// partners (pairs of halves), or 2 V neighbours; past R any 2 V neighbours.  A head
// is a group of G lanes, a power of two, with NU units each, so a head's reduction is
// log2(G) lane steps and no workgroup barrier.  A wave takes one token's next 64 / G
// heads U times: cosines, sines and weights are read once for all of them.
#include <type_traits>

#include "elem_dev.h"

namespace moeq {

namespace {

struct HeadArgs {
    moe_heads h;
    int64_t t0;         // the launch's first token
    int64_t waves;      // of this launch
    int gbits;          // lanes of a head: 1 << gbits
    int per, per_q;     // waves of a token, those of them on queries
};

// V elements at any alignment of theirs.
template <int V>
struct Part;
template <>
struct Part<8> : Raw<8> {
    __device__ __forceinline__ void get(const void* p, int dt, int64_t i) {
        load<false, true>(p, dt, i);
    }
};
template <>
struct Part<1> : Raw<1> {
    __device__ __forceinline__ void get(const void* p, int dt, int64_t i) { load(p, dt, i); }
};
typedef uint32_t u32_any __attribute__((aligned(2)));
template <>
struct Part<2> {
    uint32_t a, b;
    __device__ __forceinline__ void get(const void* p, int dt, int64_t i) {
        if (dt == MOE_DT_F32) {
            const uint32_t* q = static_cast<const uint32_t*>(p) + i;
            a = q[0];
            b = q[1];
        } else {
            a = *reinterpret_cast<const u32_any*>(static_cast<const uint16_t*>(p) + i);
            b = 0u;
        }
    }
    __device__ __forceinline__ void f32(int dt, float (&v)[2]) const {
        if (dt == MOE_DT_F32) {
            v[0] = __uint_as_float(a);
            v[1] = __uint_as_float(b);
        } else if (dt == MOE_DT_BF16) {
            v[0] = __uint_as_float(a << 16);
            v[1] = __uint_as_float(a & 0xffff0000u);
        } else {
            const f16x2 h = __builtin_bit_cast(f16x2, a);
            v[0] = (float)h[0];
            v[1] = (float)h[1];
        }
    }
};

template <int V>
__device__ __forceinline__ void put(void* p, int dt, int64_t i, const float (&v)[V]) {
    if constexpr (V == 2) {
        if (dt == MOE_DT_F32) {
            store_f32<2>(p, dt, i, v);
        } else {
            *reinterpret_cast<u32_any*>(static_cast<uint16_t*>(p) + i) =
                dt == MOE_DT_BF16 ? pack_bf16(v[0], v[1]) : pack_f16(v[0], v[1]);
        }
    } else {
        store_f32<V, false, true>(p, dt, i, v);
    }
}

template <int V, int NU, int U>
__global__ __launch_bounds__(256) void k_heads(HeadArgs A) {
    const moe_heads& P = A.h;
    const int lane = threadIdx.x & 63;
    const int64_t wv = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (wv >= A.waves) return;
    const int64_t t = A.t0 + wv / A.per;
    const int part = (int)(wv % A.per);
    const bool is_q = part < A.per_q;
    const moe_head_set& S = is_q ? P.q : P.k;
    const int G = 1 << A.gbits;
    const int hps = 64 >> A.gbits;                   // heads of a step
    const int h0 = (is_q ? part : part - A.per_q) * U * hps + (lane >> A.gbits);
    const int D = P.D, R = P.R, dt = P.dtype;
    const char* base = static_cast<const char*>(S.x);

    // this lane's units: the places of their two parts, and whether they are of the head
    int at0[NU], at1[NU];
    bool turn[NU], in0[NU], in1[NU];
#pragma unroll
    for (int n = 0; n < NU; ++n) {
        const int u = (lane & (G - 1)) + n * G;
        turn[n] = 2 * V * u < R;
        const bool halves = turn[n] && !P.interleaved;
        at0[n] = halves ? V * u : 2 * V * u;
        at1[n] = halves ? R / 2 + V * u : 2 * V * u + V;
        in0[n] = at0[n] < D;
        in1[n] = at1[n] < D;                         // V = 1: the last of an odd head
    }

    Part<V> x0[U][NU], x1[U][NU], w0[NU], w1[NU];
    int64_t row[U];
#pragma unroll
    for (int s = 0; s < U; ++s) {
        const int h = h0 + s * hps;
        row[s] = h < S.heads ? t * S.ld_t + h * S.ld_h : -1;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            if (h < S.heads && in0[n]) x0[s][n].get(base, dt, row[s] + at0[n]);
            if (h < S.heads && in1[n]) x1[s][n].get(base, dt, row[s] + at1[n]);
        }
    }
    float c[NU][V], sn[NU][V];
    if (P.pos) {
        const int64_t p = P.pos_bits == 64 ? static_cast<const int64_t*>(P.pos)[t]
                                           : static_cast<const int32_t*>(P.pos)[t];
        const bool known = p >= 0 && p < P.table_rows;
        const float* row_c = P.table + (known ? p : 0) * R;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int u = (lane & (G - 1)) + n * G;
            if (turn[n]) {
                load_f32<V, true>(row_c, MOE_DT_F32, V * u, c[n]);
                load_f32<V, true>(row_c, MOE_DT_F32, R / 2 + V * u, sn[n]);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (!turn[n]) c[n][e] = 1.f, sn[n][e] = 0.f;
                else if (!known) c[n][e] = sn[n][e] = __uint_as_float(0x7fc00000u);
            }
        }
    }
    float f0[NU][V], f1[NU][V];
    if (S.w) {
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            if (in0[n]) w0[n].get(S.w, P.w_dtype, at0[n]);
            if (in1[n]) w1[n].get(S.w, P.w_dtype, at1[n]);
        }
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            w0[n].f32(P.w_dtype, f0[n]);
            w1[n].f32(P.w_dtype, f1[n]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                f0[n][e] += P.w_offset;
                f1[n][e] += P.w_offset;
            }
        }
    }

#pragma unroll
    for (int s = 0; s < U; ++s) {
        float a[NU][V], b[NU][V];
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            x0[s][n].f32(dt, a[n]);
            x1[s][n].f32(dt, b[n]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (!in0[n] || row[s] < 0) a[n][e] = 0.f;
                if (!in1[n] || row[s] < 0) b[n][e] = 0.f;
            }
        }
        if (S.w) {
            auto mean_square = [&](float k) {
                float ss = 0.f;
#pragma unroll
                for (int n = 0; n < NU; ++n)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float p = a[n][e] * k, q = b[n][e] * k;
                        ss += p * p;
                        ss += q * q;
                    }
                for (int off = 1; off < G; off <<= 1) ss += __shfl_xor(ss, off);
                return ss / (float)D;
            };
            // 1 / sqrt(mean square + eps) of the head times k, 1 unless the squares leave
            // fp32's range: 2^-80 past its top, 2^100 where squares that underflow might
            // count.  v * k * rstd does not notice.
            float k = 1.f;
            float ms = mean_square(1.f) + P.eps;
            const bool far = !(ms >= 0x1p-100f && ms < __builtin_inff());
            if (__any(far)) {
                if (far) k = ms < 1.f ? 0x1p100f : 0x1p-80f;
                const float again = mean_square(k) + P.eps * k * k;
                if (far) ms = again;
            }
            const float rstd = 1.f / sqrtf(ms);
#pragma unroll
            for (int n = 0; n < NU; ++n)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    a[n][e] = a[n][e] * k * rstd * f0[n][e];
                    b[n][e] = b[n][e] * k * rstd * f1[n][e];
                }
        }
        if (row[s] < 0) continue;
        const int64_t out = t * S.ld_out_t + (h0 + s * hps) * S.ld_out_h;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            if (P.pos && turn[n]) {
                if (P.interleaved) {
                    // pair i at elements 2i and 2i + 1 of the unit's 2 V neighbours
                    float z[2 * V];
#pragma unroll
                    for (int e = 0; e < V; ++e) z[e] = a[n][e], z[V + e] = b[n][e];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float p = z[2 * e], q = z[2 * e + 1];
                        z[2 * e] = p * c[n][e] - q * sn[n][e];
                        z[2 * e + 1] = q * c[n][e] + p * sn[n][e];
                    }
#pragma unroll
                    for (int e = 0; e < V; ++e) a[n][e] = z[e], b[n][e] = z[V + e];
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float p = a[n][e], q = b[n][e];
                        a[n][e] = p * c[n][e] - q * sn[n][e];
                        b[n][e] = q * c[n][e] + p * sn[n][e];
                    }
                }
            }
            if (in0[n]) put<V>(S.out, dt, out + at0[n], a[n]);
            if (in1[n]) put<V>(S.out, dt, out + at1[n], b[n]);
        }
    }
}

}  // namespace

int launch_heads(const moe_heads& h, int64_t T, void* stream) {
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    HeadArgs A{h, 0, 0, 0, 0, 0};
    auto go = [&](auto v, auto nu, auto u) {
        constexpr int V = decltype(v)::value, NU = decltype(nu)::value, U = decltype(u)::value;
        const int lanes = ((h.D + 2 * V - 1) / (2 * V) + NU - 1) / NU;
        A.gbits = 0;
        while (1 << A.gbits < lanes) ++A.gbits;
        const int per_wave = (64 >> A.gbits) * U;
        A.per_q = (h.q.heads + per_wave - 1) / per_wave;
        A.per = A.per_q + (h.k.heads + per_wave - 1) / per_wave;
        const int64_t most = rows_of_launch(1) / 4 * 4 / A.per - 4;     // tokens of a launch
        for (A.t0 = 0; A.t0 < T; A.t0 += most) {
            A.waves = (T - A.t0 < most ? T - A.t0 : most) * A.per;
            k_heads<V, NU, U><<<(unsigned)((A.waves + 3) / 4), 256, 0, s>>>(A);
        }
    };
    using std::integral_constant;
    auto by_u = [&](auto v, auto nu) {
        // Every head step in a wave of its own while that leaves room on the chip; then
        // four to a wave, which share the table's row and the weights.
        constexpr int V = decltype(v)::value;
        const int64_t heads = (int64_t)h.q.heads + h.k.heads;
        if (T * heads * h.D < (int64_t)1 << 21) go(v, nu, integral_constant<int, 1>{});
        else go(v, nu, integral_constant<int, V == 8 ? 4 : 2>{});
    };
    integral_constant<int, 1> c1;
    integral_constant<int, 2> c2;
    integral_constant<int, 4> c4;
    integral_constant<int, 8> c8;
    if (h.D % 16 == 0 && h.R % 16 == 0) {
        by_u(c8, c1);
    } else if (h.D % 4 == 0 && h.R % 4 == 0) {
        if (h.D <= 256) by_u(c2, c1);
        else if (h.D <= 512) by_u(c2, c2);
        else by_u(c2, c4);
    } else {
        if (h.D <= 128) by_u(c1, c1);
        else if (h.D <= 256) by_u(c1, c2);
        else if (h.D <= 512) by_u(c1, c4);
        else by_u(c1, c8);
    }
    MOEQ_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace moeq
