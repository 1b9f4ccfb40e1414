// Products in 8-bit integers for few rows: weight-streaming skinny MFMA.
//
//   acc[r, n] = sum_k q[r, k] * W[n, k]                     (exact, int32)
//   out[r, n] = qscale[r] * wscale[n] * acc[r, n] (+ bias)  or, over
//   interleaved gate and up rows,  h[r, n] = silu(g) * u    (fp32)
//
// v_mfma_i32_16x16x64_i8 multiplies 16 weight rows (A: one 1024-byte tile, a
// contiguous 16-byte load per lane) by up to 16 token rows (B: gathered 16-byte
// loads from the caches).  The KS waves of a workgroup split the inputs and add
// their int32 sums in LDS (integer sums: any order gives the same bits).
//
// The weights' stream bounds it.  Measured (us, weights from HBM): routed
// experts, H 6144, I 2048, 8 of 256, gate/up + codes of h + down: 58 at one
// token (302 MB), 340 at 8, 926 at 32 (167 experts, 6.3 GB: 6.8 TB/s, a read alone
// reaches 6.1 to 7.0).  A skewed router costs more: an expert's workgroups stream
// its weights once for every 16 rows, one time after the other (tokens by a Zipf
// law over the experts, at 32 / 64 / 128 / 256 tokens: 615 / 989 / 1369 / 1916 us,
// 1.09 / 1.12 / 1.23 / 1.50 times the touched weights at 7.0 TB/s).
// One 6144 x 6144 matrix at one token 10.2 (38 MB), 1024 x 1024 3.5.
// Many experts stream best from one-wave workgroups (KS 1, 8 tiles in flight: on
// one routing of 32 tokens 889 us, 951 with 2 x 2 waves, 967 with KS 4); a lone
// matrix needs its inputs split to fill the chip (KS 4 with 2 row groups, 8 with
// one below 256 row groups: 6144 -> 2048 5.9 us against 8.2 with KS 4).
#include <type_traits>

#include "i8_dev.h"

namespace moeq {

namespace {

__device__ __forceinline__ i32x4 mfma_i8(u32x4 a, u32x4 b, i32x4 acc) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), acc, 0, 0, 0);
}

struct Rows {
    int e;          // expert, -1: none
    int64_t r0, m;  // its first row and its rows
};

// The s-th expert with rows, in ascending id.
__device__ __forceinline__ Rows find_rows(const I8Pass& A, int s, int lane) {
    if (!A.offsets) return Rows{0, 0, A.T};
    int seen = 0;
    for (int e0 = 0; e0 < A.E; e0 += 256) {
        const Offsets4 o = load_offsets(A.offsets, A.E, e0, lane);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint64_t m = __ballot(o.o1[c] > o.o0[c]);
            const int n = __popcll(m);
            if (s < seen + n) {
                for (int i = 0; i < s - seen; ++i) m &= m - 1;
                const int owner = uniform(__ffsll((unsigned long long)m) - 1);
                const int a = __builtin_amdgcn_readlane(o.o0[c], owner);
                return Rows{e0 + 64 * c + owner, a,
                            __builtin_amdgcn_readlane(o.o1[c], owner) - a};
            }
            seen += n;
        }
    }
    return Rows{-1, 0, 0};
}

// Codes row `src` of A.x into LDS, zeros from K to `width`; two passes over the
// row, the second from the caches.
template <int KS>
__device__ __forceinline__ void code_row(const I8Pass& A, int64_t src, int8_t* q, float* scale,
                                         uint32_t* red, int width) {
    const int tid = threadIdx.x;
    const int64_t at = src * A.ldx;
    uint32_t amax = 0u;
    auto each = [&](auto&& f) {
        if (A.x_vec8) {
            for (int h = tid * 8; h < A.K; h += KS * 64 * 8) {
                float v[8];
                load_f32<8>(A.x, A.x_dtype, at + h, v);
                f(h, v, std::integral_constant<int, 8>{});
            }
        } else {
            for (int h = tid; h < A.K; h += KS * 64) {
                float v[1];
                load_f32<1>(A.x, A.x_dtype, at + h, v);
                f(h, v, std::integral_constant<int, 1>{});
            }
        }
    };
    each([&](int, const float* v, auto n) {
#pragma unroll
        for (int e = 0; e < decltype(n)::value; ++e)
            amax = max(amax, __float_as_uint(v[e]) & 0x7fffffffu);
    });
    amax = block_max(amax, red, KS);
    const RowCode rc = row_code(amax);
    if (tid == 0) *scale = rc.scale;
    each([&](int h, const float* v, auto n) {
        if constexpr (decltype(n)::value == 8)
            *reinterpret_cast<uint2*>(q + h) =
                uint2{pack_codes4(v, rc.mul), pack_codes4(v + 4, rc.mul)};
        else
            q[h] = code1(v[0], rc.mul);
    });
    for (int h = A.K + tid; h < width; h += KS * 64) q[h] = 0;
    if constexpr (KS > 1) __syncthreads();   // red is free again
}

// A workgroup owns NG row groups of one matrix and its KS waves split the
// inputs.  U input tiles are in flight per wave: a tile's registers are
// reloaded as soon as it is multiplied.
//
// XR > 0: the rows come uncoded (A.x, of A.x_dtype) and every workgroup codes
// the XR rows it multiplies in LDS, behind its first weight loads, which saves
// a launch where there are few of them.
template <bool PAIR, int NG, int KS, int U, int XR>
__global__ __launch_bounds__(KS * 64) void k_i8(I8Pass A, int ngroups, bool quads) {
    constexpr int ROWS = XR ? XR : 16;                    // token rows of a chunk
    __shared__ int32_t sums[KS > 1 ? NG * 256 : 1];
    __shared__ float xscale[XR ? XR : 1];
    __shared__ uint32_t red[KS];
    extern __shared__ __attribute__((aligned(16))) int8_t xcodes[];   // XR rows of nkt tiles
    const int lane = threadIdx.x & 63, ks = uniform(threadIdx.x >> 6);
    const Rows r = find_rows(A, blockIdx.y, lane);
    if (r.e < 0) return;
    const int nkt = (A.K + kI8TileK - 1) / kI8TileK;      // tiles with weights
    const int g0 = blockIdx.x * NG;
    const int k0 = nkt * ks / KS, k1 = nkt * (ks + 1) / KS;
    const uint8_t* w[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g)
        w[g] = A.w + r.e * A.w_stride +
               min(g0 + g, ngroups - 1) * (i8_tiles_k(A.K) * kI8TileBytes) + lane * 16;
    const float* sw = A.wscale + r.e * A.wscale_stride;

    for (int64_t c0 = (int64_t)blockIdx.z * ROWS; c0 < r.m; c0 += (int64_t)gridDim.z * ROWS) {
        const int left = (int)min((int64_t)ROWS, r.m - c0);
        const bool in = (lane & 15) < left;
        const int64_t row = r.r0 + c0 + (in ? lane & 15 : 0);
        auto source = [&](int64_t i) {
            return A.offsets && A.perm_src ? (int64_t)(A.perm_src[i] / A.k) : i;
        };
        const int64_t src = source(row);
        const int8_t* xq = XR ? xcodes + (in ? lane & 15 : 0) * (nkt * kI8TileK)
                              : A.q + src * A.ldq;
        xq += (lane >> 4) * 16;
        u32x4 wb[U][NG], xb[U];
        auto load = [&](int u, int kt) {
            const int64_t k = min(kt, k1 - 1);
#pragma unroll
            for (int g = 0; g < NG; ++g) wb[u][g] = load_stream16(w[g] + k * kI8TileBytes);
            if constexpr (!XR) xb[u] = *reinterpret_cast<const u32x4*>(xq + k * kI8TileK);
        };
        i32x4 acc[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) acc[g] = i32x4{0, 0, 0, 0};
        if (k0 < k1) {
#pragma unroll
            for (int u = 0; u < U; ++u) load(u, k0 + u);
        }
        if constexpr (XR > 0) {
            for (int i = 0; i < left; ++i)
                code_row<KS>(A, source(r.r0 + c0 + i), xcodes + i * (nkt * kI8TileK), xscale + i,
                             red, nkt * kI8TileK);
            __syncthreads();
        }
        if (k0 < k1) {
            for (int kt = k0; kt < k1; kt += U) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (kt + u < k1) {
                        if constexpr (XR > 0)
                            xb[u] = *reinterpret_cast<const u32x4*>(xq + (kt + u) * kI8TileK);
#pragma unroll
                        for (int g = 0; g < NG; ++g) acc[g] = mfma_i8(wb[u][g], xb[u], acc[g]);
                    }
                    load(u, kt + u + U);
                }
            }
        }
        if constexpr (KS > 1) {
            // int32 sums over the input parts: the same bits in any order
            if (ks == 0) {
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sums[(g * 4 + i) * 64 + lane] = acc[g][i];
            }
            __syncthreads();
            if (ks > 0) {
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        __hip_atomic_fetch_add(&sums[(g * 4 + i) * 64 + lane], acc[g][i],
                                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            }
            __syncthreads();
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[g][i] = sums[(g * 4 + i) * 64 + lane];
        }
        if (in) {
            const Scale sq = split(XR ? xscale[lane & 15] : A.qscale[src]);
#pragma unroll
            for (int g = 0; g < NG; g += PAIR ? 2 : 1) {
                // one wave writes a row group
                if (g / (PAIR ? 2 : 1) % KS != ks || g0 + g >= ngroups) continue;
                const int ch = (g0 + g) / (PAIR ? 2 : 1) * 16 + (lane >> 4) * 4;
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = min(ch + i, A.N - 1);
                    if constexpr (PAIR)
                        y[i] = silu_mul(scaled(sq, split(sw[c]), acc[g][i]),
                                        scaled(sq, split(sw[A.N + c]), acc[g + 1][i]));
                    else
                        y[i] = scaled(sq, split(sw[c]), acc[g][i]) + (A.bias ? A.bias[c] : 0.f);
                }
                const int64_t at = row * A.ld_out + ch;
                if (quads) {
                    if (ch < A.N) store_quad(A.out, A.out_dtype, at, y);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float y1[1] = {y[i]};
                        if (ch + i < A.N) store_f32<1>(A.out, A.out_dtype, at + i, y1);
                    }
                }
            }
        }
        if constexpr (KS > 1 || XR > 0) __syncthreads();   // before the next chunk
    }
}

template <bool PAIR, int NG, int KS, int U, int XR>
void launch(const I8Pass& p, int ngroups, int64_t slots, int64_t mean, hipStream_t s) {
    const uintptr_t four = p.out_dtype == MOE_DT_F32 ? 16 : 8;
    const bool quads = p.N % 4 == 0 && p.ld_out % 4 == 0 &&
                       reinterpret_cast<uintptr_t>(p.out) % four == 0;
    // a workgroup takes its matrix's chunks of rows in turn
    constexpr int ROWS = XR ? XR : 16;
    const dim3 grid((unsigned)((ngroups + NG - 1) / NG), (unsigned)slots,
                    (unsigned)((mean + ROWS - 1) / ROWS));
    k_i8<PAIR, NG, KS, U, XR><<<grid, KS * 64, XR * round_up(p.K, kI8TileK), s>>>(p, ngroups,
                                                                                 quads);
}

template <bool PAIR, int XR>
void pick(const I8Pass& p, int ngroups, int64_t slots, int64_t mean, hipStream_t s) {
    const int64_t all = slots * ngroups;
    if (all >= 1024) launch<PAIR, 2, 1, 8, XR>(p, ngroups, slots, mean, s);
    else if (all >= 256) launch<PAIR, 2, 4, 8, XR>(p, ngroups, slots, mean, s);
    else launch<PAIR, PAIR ? 2 : 1, 8, 4, XR>(p, ngroups, slots, mean, s);
}

}  // namespace

// (One matrix of 6144 x 6144 at one token: 9.1 us against 10.6 with the codes
// made by a launch of their own.  Routed experts do not: every expert's
// workgroups would code its rows, 60.4 against 58.0 us at one token.)
bool i8_codes_itself(int64_t T, int32_t K, bool routed) {
    return !routed && T <= 4 && T * round_up(K, kI8TileK) <= 24576;
}

int launch_i8(const I8Pass& p, bool pair, void* stream) {
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int64_t rows = p.T * p.k, slots = p.offsets ? (p.E < rows ? p.E : rows) : 1;
    const int64_t mean = rows / slots + (rows % slots != 0);    // rows of a matrix
    const int ngroups = (int)(round_up(p.N, 16) / 16) * (pair ? 2 : 1);
    if (p.x) {
        const bool one = p.T == 1;
        if (one && pair) pick<true, 1>(p, ngroups, slots, mean, s);
        else if (one) pick<false, 1>(p, ngroups, slots, mean, s);
        else if (pair) pick<true, 4>(p, ngroups, slots, mean, s);
        else pick<false, 4>(p, ngroups, slots, mean, s);
    } else {
        // More rows go to the GEMM: from 17 of one matrix, unless this kernel's
        // workgroups, one for every 16 rows, find a CU each (us here / there:
        // 6144 -> 4096 at 32 rows 12.2 / 15.5, at 33 18.0 / 14.2; 6144 -> 256 at 200
        // rows 7.3 / 9.7; 6144 x 6144 at 32 21.2 / 17.1); from 13 of an expert on
        // average, since experts differ.
        const int ng = pair || slots * ngroups >= 256 ? 2 : 1;     // as pick() has it
        const int64_t wgs = (ngroups + ng - 1) / ng * ((mean + 15) / 16);
        if (slots > 1 ? mean > 12 : mean > 16 && wgs > 256)
            return launch_gemm_i8(p, pair, stream);
        if (pair) pick<true, 0>(p, ngroups, slots, mean, s);
        else pick<false, 0>(p, ngroups, slots, mean, s);
    }
    MOEQ_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace moeq
