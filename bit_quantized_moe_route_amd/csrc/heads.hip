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
// log2(G) lane steps and no workgroup barrier; a wave holds 64 / G heads of one token.
//
// HBM bounds large batches: 4096 tokens of 64 + 8 heads of 128 in bf16 move 151 MB in
// 30 us (5.0 TB/s; a plain copy reaches 5.1 to 5.8).  A wave with several steps of heads,
// which read the table's row and the weights once, was no faster (1 / 2 / 4 / 8 steps:
// 32 / 32.9 / 33.1 / 39 us).  One token is a launch and the chain position -> table -> rotation: 3.6 us.
#include <type_traits>

#include "elem_dev.h"

namespace moeq {

namespace {

struct HeadArgs {
    moe_heads h;
    int64_t t0;         // the launch's first token
    int gbits;          // lanes of a head: 1 << gbits
    int per, per_q;     // waves of a token, those of them on queries
};

typedef uint32_t u32_any __attribute__((aligned(2)));

// V elements of type DT at any alignment of theirs, as loaded.
template <int V, int DT>
struct Part {
    static constexpr int W = DT == MOE_DT_F32 ? V : (V + 1) / 2;      // words
    uint32_t w[W];
    __device__ __forceinline__ void get(const char* p, int i) {
        const char* q = p + i * (DT == MOE_DT_F32 ? 4 : 2);
        if constexpr (V == 8) {
#pragma unroll
            for (int k = 0; k < W; k += 4) {
                const u32x4 u = load16<false, true>(q + 4 * k);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[k + e] = u[e];
            }
        } else if constexpr (DT != MOE_DT_F32 && V == 1) {
            w[0] = *reinterpret_cast<const uint16_t*>(q);
        } else {
#pragma unroll
            for (int k = 0; k < W; ++k) w[k] = reinterpret_cast<const u32_any*>(q)[k];
        }
    }
    __device__ __forceinline__ void f32(float (&v)[V]) const {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if constexpr (DT == MOE_DT_F32) {
                v[e] = __uint_as_float(w[e]);
            } else if constexpr (DT == MOE_DT_BF16) {
                v[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
            } else {
                v[e] = (float)__builtin_bit_cast(f16x2, w[e / 2])[e & 1];
            }
        }
    }
};

template <int V, int DT, bool STREAM>
__device__ __forceinline__ void put(char* p, int i, const float (&v)[V]) {
    char* q = p + i * (DT == MOE_DT_F32 ? 4 : 2);
    if constexpr (V == 2 && DT != MOE_DT_F32) {
        *reinterpret_cast<u32_any*>(q) =
            DT == MOE_DT_BF16 ? pack_bf16(v[0], v[1]) : pack_f16(v[0], v[1]);
    } else {
        store_f32<V, STREAM, true>(q, DT, 0, v);
    }
}

// STREAM: results past the caches.
template <int DT, int V, int NU, bool STREAM>
__global__ __launch_bounds__(256) void k_heads(HeadArgs A) {
    constexpr int B = DT == MOE_DT_F32 ? 4 : 2;
    const moe_heads& P = A.h;
    const int lane = threadIdx.x & 63;
    const int64_t t = A.t0 + blockIdx.x;
    const int part = (int)(blockIdx.y * (blockDim.x >> 6)) +
                     __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (part >= A.per) return;
    const bool is_q = part < A.per_q;
    const moe_head_set& S = is_q ? P.q : P.k;
    const int G = 1 << A.gbits;
    const int h = (is_q ? part : part - A.per_q) * (64 >> A.gbits) + (lane >> A.gbits);
    const int D = P.D, R = P.R;
    const char* x = static_cast<const char*>(S.x) + t * S.ld_t * B;
    char* out = static_cast<char*>(S.out) + t * S.ld_out_t * B;

    // This lane's units: the places of their two parts, and whether they are of the head.
    // Those that are not read another's (and heads past the last the last one's), unused.
    int at0[NU], at1[NU], unit[NU];
    bool turn[NU], in0[NU], in1[NU];
#pragma unroll
    for (int n = 0; n < NU; ++n) {
        const int u = (lane & (G - 1)) + n * G;
        unit[n] = 2 * V * u < D ? u : 0;
        turn[n] = 2 * V * unit[n] < R;
        const bool halves = turn[n] && !P.interleaved;
        at0[n] = halves ? V * unit[n] : 2 * V * unit[n];
        at1[n] = halves ? R / 2 + V * unit[n] : 2 * V * unit[n] + V;
        in0[n] = 2 * V * u < D;
        in1[n] = in0[n] && at1[n] < D;               // V = 1: the last of an odd head
        if (V == 1 && at1[n] >= D) at1[n] = at0[n];
    }

    Part<V, DT> x0[NU], x1[NU];
    const char* row = x + (int64_t)min(h, S.heads - 1) * S.ld_h * B;
#pragma unroll
    for (int n = 0; n < NU; ++n) {
        x0[n].get(row, at0[n]);
        x1[n].get(row, at1[n]);
    }
    float c[NU][V], sn[NU][V];
    if (P.pos) {
        const int64_t p = P.pos_bits == 64 ? static_cast<const int64_t*>(P.pos)[t]
                                           : static_cast<const int32_t*>(P.pos)[t];
        const bool known = p >= 0 && p < P.table_rows;
        const float* row_c = P.table + (known ? p : 0) * R;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int i = turn[n] ? V * unit[n] : 0;
            load_f32<V, true>(row_c, MOE_DT_F32, i, c[n]);
            load_f32<V, true>(row_c, MOE_DT_F32, R / 2 + i, sn[n]);
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
            load_f32<V, true>(S.w, P.w_dtype, at0[n], f0[n]);
            load_f32<V, true>(S.w, P.w_dtype, at1[n], f1[n]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                f0[n][e] += P.w_offset;
                f1[n][e] += P.w_offset;
            }
        }
    }

    float a[NU][V], b[NU][V];
#pragma unroll
    for (int n = 0; n < NU; ++n) {
        x0[n].f32(a[n]);
        x1[n].f32(b[n]);
    }
    if (S.w) {
        auto mean_square = [&](float k) {
            float ss = 0.f;
#pragma unroll
            for (int n = 0; n < NU; ++n)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float p = in0[n] ? a[n][e] * k : 0.f, q = in1[n] ? b[n][e] * k : 0.f;
                    ss += p * p;
                    ss += q * q;
                }
            for (int off = 1; off < G; off <<= 1) ss += __shfl_xor(ss, off);
            return ss / (float)D;
        };
        const float ms = mean_square(1.f) + P.eps;
        const bool far = !(ms >= 0x1p-100f && ms < __builtin_inff());
        float rstd = 1.f / sqrtf(ms);
        if (__any(far)) {
            // Where the squares leave fp32's range, the head times k: 2^-80 past its top,
            // 2^100 where squares that underflow might count.  v goes up before it meets its
            // 1 / sqrt(mean square + eps), and down after it, so that neither end is lost.
            const float up = far && ms < 1.f ? 0x1p100f : 1.f;
            const float down = far && up == 1.f ? 0x1p-80f : 1.f, k = up * down;
            const float again = mean_square(k) + P.eps * k * k;
            const float r = far ? 1.f / sqrtf(again) : 1.f;
            if (far) rstd = 1.f;
#pragma unroll
            for (int n = 0; n < NU; ++n)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    a[n][e] = a[n][e] * up * r * down;
                    b[n][e] = b[n][e] * up * r * down;
                }
        }
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                a[n][e] = a[n][e] * rstd * f0[n][e];
                b[n][e] = b[n][e] * rstd * f1[n][e];
            }
    }
    if (h >= S.heads) return;
    char* to = out + (int64_t)h * S.ld_out_h * B;
#pragma unroll
    for (int n = 0; n < NU; ++n) {
        if (P.pos) {
            float z[2 * V];
#pragma unroll
            for (int e = 0; e < V; ++e) z[e] = a[n][e], z[V + e] = b[n][e];
            if (P.interleaved) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float p = z[2 * e], q = z[2 * e + 1];
                    z[2 * e] = p * c[n][e] - q * sn[n][e];
                    z[2 * e + 1] = q * c[n][e] + p * sn[n][e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float p = z[e], q = z[V + e];
                    z[e] = p * c[n][e] - q * sn[n][e];
                    z[V + e] = q * c[n][e] + p * sn[n][e];
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                a[n][e] = turn[n] ? z[e] : a[n][e];
                b[n][e] = turn[n] ? z[V + e] : b[n][e];
            }
        }
        if (in0[n]) put<V, DT, STREAM>(to, at0[n], a[n]);
        if (in1[n]) put<V, DT, STREAM>(to, at1[n], b[n]);
    }
}

}  // namespace

int launch_heads(const moe_heads& h, int64_t T, void* stream) {
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    HeadArgs A{h, 0, 0, 0, 0};
    using std::integral_constant;
    auto go = [&](auto dt, auto v, auto nu, auto st) {
        constexpr int V = decltype(v)::value, NU = decltype(nu)::value;
        const int lanes = ((h.D + 2 * V - 1) / (2 * V) + NU - 1) / NU;
        A.gbits = 0;
        while (1 << A.gbits < lanes) ++A.gbits;
        const int per_wave = 64 >> A.gbits;
        A.per_q = (h.q.heads + per_wave - 1) / per_wave;
        A.per = A.per_q + (h.k.heads + per_wave - 1) / per_wave;
        // a token's waves, up to four a workgroup
        const int groups = (A.per + 3) / 4, waves = (A.per + groups - 1) / groups;
        const int64_t most = rows_of_launch(waves) / groups;     // tokens of a launch
        for (A.t0 = 0; A.t0 < T; A.t0 += most) {
            const dim3 grid((unsigned)(T - A.t0 < most ? T - A.t0 : most), (unsigned)groups);
            k_heads<decltype(dt)::value, V, NU, decltype(st)::value><<<grid, waves * 64, 0, s>>>(A);
        }
    };
    // Results of 2M elements and more go past the caches, as the block norms' do (4096
    // tokens of 72 heads of 128: 42.0 -> 33.1 us).
    const bool large = T * ((int64_t)h.q.heads + h.k.heads) * h.D >= (int64_t)1 << 21;
    integral_constant<int, 1> c1;
    integral_constant<int, 2> c2;
    integral_constant<int, 4> c4;
    integral_constant<int, 8> c8;
    auto by_type = [&](auto dt) {
        auto by = [&](auto v, auto nu) { go(dt, v, nu, std::false_type{}); };
        if (h.D % 16 == 0 && h.R % 16 == 0) {
            if (large) go(dt, c8, c1, std::true_type{});
            else by(c8, c1);
        } else if (h.D % 4 == 0 && h.R % 4 == 0) {
            if (h.D <= 256) by(c2, c1);
            else if (h.D <= 512) by(c2, c2);
            else by(c2, c4);
        } else {
            if (h.D <= 128) by(c1, c1);
            else if (h.D <= 256) by(c1, c2);
            else if (h.D <= 512) by(c1, c4);
            else by(c1, c8);
        }
    };
    if (h.dtype == MOE_DT_F32) by_type(integral_constant<int, MOE_DT_F32>{});
    else if (h.dtype == MOE_DT_BF16) by_type(integral_constant<int, MOE_DT_BF16>{});
    else by_type(integral_constant<int, MOE_DT_F16>{});
    MOEQ_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace moeq
