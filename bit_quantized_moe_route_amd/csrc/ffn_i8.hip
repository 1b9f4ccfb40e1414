// Products in 8-bit integers for few rows: weight-streaming skinny MFMA.
//
//   acc[r, n] = sum_k q[r, k] * W[n, k]                     (exact, int32)
//   out[r, n] = qscale[r] * wscale[n] * acc[r, n] (+ bias)  or, over
//   interleaved gate and up rows,  h[r, n] = silu(g) * u    (fp32)
//
// v_mfma_i32_16x16x64_i8 multiplies 16 weight rows (A: one 1024-byte tile, a
// 16-byte load per lane) by up to 16 token rows (B: gathered 16-byte loads
// from the caches).  The KS waves of a workgroup split the inputs and add
// their int32 sums in LDS (integer sums: any order gives the same bits).
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
    for (int e0 = 0; e0 < A.E; e0 += 64) {
        const int e = e0 + lane;
        const int o0 = e < A.E ? A.offsets[e] : 0;
        const int o1 = e < A.E ? A.offsets[e + 1] : 0;
        uint64_t m = __ballot(o1 > o0);
        const int n = __popcll(m);
        if (s < seen + n) {
            for (int i = 0; i < s - seen; ++i) m &= m - 1;
            const int owner = __ffsll((unsigned long long)m) - 1;
            const int a = __shfl(o0, owner), b = __shfl(o1, owner);
            return Rows{e0 + owner, a, b - a};
        }
        seen += n;
    }
    return Rows{-1, 0, 0};
}

template <bool PAIR, int NG, int KS>
__global__ __launch_bounds__(KS * 64) void k_i8(I8Pass A, int ngroups) {
    __shared__ i32x4 part[KS][NG][64];
    const int lane = threadIdx.x & 63, ks = threadIdx.x >> 6;
    const Rows rw = find_rows(A, blockIdx.y, lane);
    if (rw.e < 0) return;
    const int nkt = (A.K + kI8TileK - 1) / kI8TileK;      // tiles with weights
    const int64_t gbytes = i8_tiles_k(A.K) * kI8TileBytes;
    const int g0 = blockIdx.x * NG;
    const uint8_t* w[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g)
        w[g] = A.w + rw.e * A.w_stride + min(g0 + g, ngroups - 1) * gbytes +
               lane * 16;
    const float* sw = A.wscale + rw.e * A.wscale_stride;
    const int k0 = (int)((int64_t)nkt * ks / KS), k1 = (int)((int64_t)nkt * (ks + 1) / KS);

    for (int64_t c0 = (int64_t)blockIdx.z * 16; c0 < rw.m; c0 += (int64_t)gridDim.z * 16) {
        const bool in = c0 + (lane & 15) < rw.m;
        const int64_t row = rw.r0 + (in ? c0 + (lane & 15) : c0);
        const int64_t src = A.offsets && A.perm_src ? A.perm_src[row] / A.k : row;
        const int8_t* xq = A.q + src * A.ldq + (lane >> 4) * 16;
        i32x4 acc[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) acc[g] = i32x4{0, 0, 0, 0};
        for (int kt = k0; kt < k1; ++kt) {
            const u32x4 b = *reinterpret_cast<const u32x4*>(xq + (int64_t)kt * kI8TileK);
#pragma unroll
            for (int g = 0; g < NG; ++g)
                acc[g] = mfma_i8(load_stream16(w[g] + (int64_t)kt * kI8TileBytes), b, acc[g]);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) part[ks][g][lane] = acc[g];
        __syncthreads();
        if (ks == 0 && in) {
#pragma unroll
            for (int g = 0; g < NG; ++g)
                for (int i = 1; i < KS; ++i) acc[g] += part[i][g][lane];
            const float sq = A.qscale[src];
            if constexpr (PAIR) {
#pragma unroll
                for (int g = 0; g < NG; g += 2) {
                    const int ch = (g0 + g) / 2 * 16 + (lane >> 4) * 4;
                    float* h = static_cast<float*>(A.out) + row * A.ld_out;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (g0 + g < ngroups && ch + i < A.N)
                            h[ch + i] = silu_mul(sq * sw[ch + i] * (float)acc[g][i],
                                                 sq * sw[A.N + ch + i] * (float)acc[g + 1][i]);
                }
            } else {
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const int ch = (g0 + g) * 16 + (lane >> 4) * 4;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (g0 + g < ngroups && ch + i < A.N) {
                            const float b = A.bias ? A.bias[ch + i] : 0.f;
                            const float y[1] = {sq * sw[ch + i] * (float)acc[g][i] + b};
                            store_f32<1>(A.out, A.out_dtype, row * A.ld_out + ch + i, y);
                        }
                }
            }
        }
        __syncthreads();
    }
}

}  // namespace

int launch_i8(const I8Pass& p, bool pair, void* stream) {
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if ((p.offsets ? p.T * p.k / p.E : p.T) > 16) return launch_gemm_i8(p, pair, stream);
    const int ngroups = (int)(round_up(p.N, 16) / 16) * (pair ? 2 : 1);
    const int64_t slots = p.offsets ? (p.E < p.T * p.k ? p.E : p.T * p.k) : 1;
    // a workgroup takes its matrix's 16-row chunks in turn
    const int64_t rows = p.offsets ? p.T * p.k / p.E : p.T;
    const dim3 grid((unsigned)((ngroups + 1) / 2), (unsigned)slots, (unsigned)(rows / 16 + 1));
    if (pair) k_i8<true, 2, 4><<<grid, 256, 0, s>>>(p, ngroups);
    else k_i8<false, 2, 4><<<grid, 256, 0, s>>>(p, ngroups);
    MOEQ_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace moeq
