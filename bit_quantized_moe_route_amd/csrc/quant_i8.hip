// The 8-bit code of rows (a scale per row) and the device layout of 8-bit
// weight matrices.
//
// Row t of x [T, K]:  a = max_k |x[t, k]|,  scale[t] = a / 127,
// q[t, k] = rint(127 x[t, k] / a).  One pass over x: a row stays in
// registers (NCH chunks of V elements per thread) between its maximum and its
// codes; rows past that (NCH = 0) are read a second time, from L2.  Bound by
// HBM: 4096 x 6144 bf16 to codes, 75 MB, in 22 us; the fp32 middle rows of a
// routed prefill batch (32768 x 2048), 336 MB, in 57 us; 4096 x 6145, whose rows
// start off 16 bytes, in 25 (39 element by element).
#include <type_traits>

#include "elem_dev.h"

namespace moeq {

namespace {

struct QuantArgs {
    const void* x;
    int64_t ldx, ldq, T, t0;   // t0: the launch's first row
    int8_t* q;
    float* scale;
    int dt, K, nw;   // nw: waves of a row
};

// Codes of elements lo .. V - 1 of a chunk at h (lo 0: all, on 8 bytes).
template <int V>
__device__ __forceinline__ void store_codes(int8_t* q, int h, const float (&v)[V], double mul,
                                            int lo) {
    if (V == 8 && lo == 0) {
        const uint2 u = {pack_codes4(&v[0], mul), pack_codes4(&v[V / 2], mul)};
        *reinterpret_cast<uint2*>(q + h) = u;
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e >= lo) q[h + e] = code1(v[e], mul);
    }
}

// ANY: rows that start off 16 bytes or end inside a chunk; the last chunk then
// ends at the row's end and shares `lo` elements with the one before.
template <int V, int NCH, bool ANY>
__global__ __launch_bounds__(1024) void k_quantize(QuantArgs A) {
    __shared__ uint32_t red[16];
    const int tid = threadIdx.x, nt = A.nw * 64;
    const int64_t t = A.t0 + blockIdx.x;
    int8_t* q = A.q + t * A.ldq;
    uint32_t amax = 0u;
    auto at = [&](int h) { return ANY ? min(h, A.K - V) : h; };
    if constexpr (NCH > 0) {
        float v[NCH][V];
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int h = (c * nt + tid) * V;
            if (h < A.K) {
                load_f32<V, ANY>(A.x, A.dt, t * A.ldx + at(h), v[c]);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) v[c][e] = 0.f;
            }
        }
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int e = 0; e < V; ++e) amax = max(amax, __float_as_uint(v[c][e]) & 0x7fffffffu);
        amax = block_max(amax, red, A.nw);
        const RowCode rc = row_code(amax);
        if (tid == 0) A.scale[t] = rc.scale;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int h = (c * nt + tid) * V;
            if (h < A.K) store_codes<V>(q, at(h), v[c], rc.mul, h - at(h));
        }
    } else {
        for (int h = tid * V; h < A.K; h += nt * V) {
            float v[V];
            load_f32<V, ANY>(A.x, A.dt, t * A.ldx + at(h), v);
#pragma unroll
            for (int e = 0; e < V; ++e) amax = max(amax, __float_as_uint(v[e]) & 0x7fffffffu);
        }
        amax = block_max(amax, red, A.nw);
        const RowCode rc = row_code(amax);
        if (tid == 0) A.scale[t] = rc.scale;
        for (int h = tid * V; h < A.K; h += nt * V) {
            float v[V];
            load_f32<V, ANY>(A.x, A.dt, t * A.ldx + at(h), v);
            store_codes<V>(q, at(h), v, rc.mul, h - at(h));
        }
    }
    const int pad = (A.K + kI8TileK - 1) / kI8TileK * kI8TileK - A.K;
    if (tid < pad) q[A.K + tid] = 0;
}

// Codes [N, K] (row-major, rows ld bytes apart) into 16-row x 64-input tiles
// of 1024 bytes, lane L's 16 bytes = row L & 15, inputs (L >> 4) * 16 .. +16;
// row group g of the matrix is group g0 + g * step of the destination.  A
// wave writes one tile; rows and inputs past the matrix are zero codes.
__global__ __launch_bounds__(256) void k_pack_i8(const int8_t* __restrict__ src, int64_t ld, int N,
                                                 int K, int nkt, int64_t ntiles, int g0, int step,
                                                 uint8_t* __restrict__ dst) {
    const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (tile >= ntiles) return;
    const int lane = threadIdx.x & 63;
    const int64_t g = tile / nkt;
    const int kt = (int)(tile % nkt);
    const int64_t n = g * 16 + (lane & 15);
    const int k = kt * kI8TileK + (lane >> 4) * 16;
    u32x4 u = {0u, 0u, 0u, 0u};
    if (n < N) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (k + i < K) u[i >> 2] |= (uint32_t)(uint8_t)src[n * ld + k + i] << (8 * (i & 3));
    }
    *reinterpret_cast<u32x4*>(dst + ((g0 + g * step) * nkt + kt) * kI8TileBytes + lane * 16) = u;
}

template <int V, bool ANY>
void launch_q(QuantArgs A, hipStream_t s) {
    const int nch = (A.K + V - 1) / V;
    auto waves = [&](int per) { return (nch + 64 * per - 1) / (64 * per); };
    auto go = [&](auto tag, int per) {
        constexpr int NCH = decltype(tag)::value;
        A.nw = per ? waves(per) : 16;
        const int64_t most = rows_of_launch(A.nw);
        for (A.t0 = 0; A.t0 < A.T; A.t0 += most) {
            const int64_t n = A.T - A.t0 < most ? A.T - A.t0 : most;
            k_quantize<V, NCH, ANY><<<(unsigned)n, A.nw * 64, 0, s>>>(A);
        }
    };
    if (V == 1 || waves(1) <= 16) go(std::integral_constant<int, 1>{}, 1);
    else if (waves(4) <= 16) go(std::integral_constant<int, V == 8 ? 4 : 1>{}, 4);
    else go(std::integral_constant<int, V == 8 ? 0 : 1>{}, 0);
}

}  // namespace

int launch_quantize_i8(const void* x, int dt, int64_t ldx, int64_t T, int32_t K, int8_t* q,
                       int64_t ldq, float* scale, bool vec8, void* stream) {
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    QuantArgs A{x, ldx, ldq, T, 0, q, scale, dt, K, 1};
    if (vec8) launch_q<8, false>(A, s);
    else if (K >= 8) launch_q<8, true>(A, s);
    else launch_q<1, false>(A, s);
    MOEQ_CHECK_LAUNCH();
    return MOE_OK;
}

int launch_pack_i8(const int8_t* codes, int64_t ld, int32_t N, int32_t K, int g0, int step,
                   void* packed, void* stream) {
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int64_t nkt = i8_tiles_k(K);
    const int64_t ntiles = round_up(N, 16) / 16 * nkt;
    k_pack_i8<<<(unsigned)((ntiles + 3) / 4), 256, 0, s>>>(codes, ld, N, K, (int)nkt, ntiles, g0,
                                                           step, static_cast<uint8_t*>(packed));
    MOEQ_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace moeq
