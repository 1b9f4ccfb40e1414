// Low-rank adapters of many requests beside a projection that they share:
//
//   h[t] = s_a * x_scale[t] * A_a x[t]           (rank r_a, fp32)
//   out[t] = y[t] + B_a h[t]                     (one rounding to y's type)
//
// a the adapter of token t's request.  Tokens go in tiles of up to 16 or 64 of one
// adapter (the plan of a batch).  Two launches, so that both products spread over the
// chip: the shrink makes h, a workgroup for a tile's tokens and, where there are few, a
// part of the inputs and a rank tile; the expand (apply) adds B h to 64 channels of y at
// a time.  h's sum is cut into chains of 128 inputs; slot s of 16 sums chains s, s + 16,
// .., and the slots join in pairs, then in fours (parts), then in order, in every kernel,
// so a token's bits depend on nothing but its row and its adapter.
//
// Both products are matrix instructions on 16-bit operands with fp32 sums.  x and the
// weights are 16-bit as they are (8-bit codes are exact in either type).  h stays fp32-like:
// it enters the second product as the sum of two numbers of the weights' type.  bf16 holds
// 16 bits of h so, enough for a 16-bit result, and a third number follows where y is fp32.
// fp16 holds 22 bits, down to its smallest step of 2^-24: so a token's row of h first goes to
// a largest of [2^14, 2^15) by a power of two, and what is 2^-17 of that still has its 22.
//
// Few tokens are bound by latency: one token, 6144 -> 6144, rank 16: 3.3 and 3.8 us for the
// two; 64 tokens and as many slots of ranks to 64, 6144 -> 2048: 7.6 and 4.7.  4096 tokens,
// 8 slots, 6144 -> 6144: 31.5 for the first (1.6 TB/s of x; every 32 tokens read their A
// from an L2) and 32.5 for the second (3.2 TB/s; a copy in its structure takes 26).
#include <type_traits>

#include "elem_dev.h"

namespace moeq {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kKt = kAdChain / 32;              // input tiles of a chain
constexpr int kSlots = kAdParts * kAdWaves;
constexpr int kWideTiles = 8;                   // rank tiles of the kernels for many tokens

struct AdArgs {
    moe_adapters S;
    const void* x;
    int64_t ldx;
    const float* x_scale;
    const int32_t* plan;
    float* h;                   // few tokens: [parts][T][rt * 16]
    u32x4* hh;                  // many: [16 tokens][rank tile][64 lanes], see k_shrink_wide
    uint2* h3;                  // ... the third numbers, if they are wanted
    float* hf;                  // ... the powers of two, [16 tokens][16]
    const void* y;
    void* out;
    int64_t ldy, ldo;
    int64_t T, tiles, pieces;   // pieces: workgroups' worth of tokens
    int64_t items0, items;      // workgroups: of earlier launches, in all
    int rec, sub;               // int32 of a record; pieces (waves' worth of tokens) of a tile
    int rt, kt, chains, full;   // rank tiles, input tiles, chains of a row, those that x fills
    int parts;
    int groups, per, cgs;       // groups of 64 channels, of a workgroup, such shares of a row
};

// Workgroup b of n in an order that gives each of the 8 XCDs, which take workgroups in
// turn, one contiguous range: items that share weights share an L2.
__device__ __forceinline__ int64_t by_xcd(int64_t b, int64_t n) {
    const int64_t q = n >> 3, r = n & 7, x = b & 7;
    return x * q + min(x, r) + (b >> 3);
}

// D += A * B over a 16 x 16 x 32 tile; operands as eight 16-bit values a lane.
template <bool BF>
__device__ __forceinline__ f32x4 mma32(u32x4 a, u32x4 b, f32x4 acc) {
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
    else
        return mfma16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), acc);
}

// The same over 16 x 16 x 16: lane L holds inner values (L >> 4) * 4 .. + 3.
template <bool BF>
__device__ __forceinline__ f32x4 mma16(uint2 a, uint2 b, f32x4 acc) {
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, a),
                                                         __builtin_bit_cast(s16x4, b), acc, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(f16x4, a),
                                                     __builtin_bit_cast(f16x4, b), acc, 0, 0, 0);
}

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return BF ? pack_bf16(lo, hi) : pack_f16(lo, hi);
}

// ---------------------------------------------------------------- the first product

// Eight inputs of a row as loaded, and as the weights' type.
template <bool BF, bool I8>
struct RawX {
    std::conditional_t<I8, uint2, u32x4> r;
    __device__ __forceinline__ void load(const char* row, int k) {
        if constexpr (I8) r = *reinterpret_cast<const uint2*>(row + k);
        else r = load16<false, true>(row + 2 * k);
    }
    // at the end of a row of K: zeros past it (codes: rows are padded with zeros to 64)
    __device__ __forceinline__ void load_end(const char* row, int k, int K) {
        if constexpr (I8) {
            r = uint2{0u, 0u};
            if (k < K) r = *reinterpret_cast<const uint2*>(row + k);
        } else {
            r = u32x4{0u, 0u, 0u, 0u};
            const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
            if (k + 8 <= K) {
                r = load16<false, true>(p + k);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (k + e < K) r[e >> 1] |= (uint32_t)p[k + e] << (16 * (e & 1));
            }
        }
    }
    __device__ __forceinline__ u32x4 get() const {
        if constexpr (I8) {
            u32x4 o;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t w = p < 2 ? r.x : r.y;
                const int sh = (p & 1) * 16;
                o[p] = pack2<BF>((float)(int8_t)(w >> sh), (float)(int8_t)(w >> (sh + 8)));
            }
            return o;
        } else {
            return r;
        }
    }
};

// The sums of one or two neighbouring slots (NS) of M x 16 tokens and RTW rank tiles.  w:
// this lane's place in the first rank tile; the rank tiles w_step apart.
template <bool BF, bool I8, int NS, int M, int RTW>
struct Slots {
    f32x4 acc[NS][RTW][M];
    RawX<BF, I8> x[kKt][M];
    u32x4 wt[kKt][RTW];

    __device__ __forceinline__ void weights(const uint8_t* w, int64_t w_step, int last, int c,
                                            int i) {
#pragma unroll
        for (int r = 0; r < RTW; ++r)
            wt[i][r] = *reinterpret_cast<const u32x4*>(w + min(r, last) * w_step +
                                                       ((int64_t)c * kKt + i) * 1024);
    }
    __device__ __forceinline__ void load(const char* const (&row)[M], const uint8_t* w,
                                         int64_t w_step, int last, int c, int i, int kl) {
        weights(w, w_step, last, c, i);
#pragma unroll
        for (int m = 0; m < M; ++m) x[i][m].load(row[m], (c * kKt + i) * 32 + kl);
    }
    __device__ __forceinline__ void mul(int s, int i) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const u32x4 v = x[i][m].get();
#pragma unroll
            for (int r = 0; r < RTW; ++r) acc[s][r][m] = mma32<BF>(wt[i][r], v, acc[s][r][m]);
        }
    }
    // The loads of the first chain; run() goes on from there.
    __device__ __forceinline__ void start(const AdArgs& A, const char* const (&row)[M],
                                          const uint8_t* w, int64_t w_step, int last, int slot,
                                          int kl) {
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int r = 0; r < RTW; ++r)
#pragma unroll
                for (int m = 0; m < M; ++m) acc[s][r][m] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (slot + NS <= A.full) {
#pragma unroll
            for (int i = 0; i < kKt; ++i) load(row, w, w_step, last, slot, i, kl);
        }
    }
    __device__ __forceinline__ void run(const AdArgs& A, const char* const (&row)[M],
                                        const uint8_t* w, int64_t w_step, int last, int slot,
                                        int kl) {
        int c = slot;
        // An input tile's registers take the next chain's as soon as they are used (at the
        // end a chain that is there, for nothing).
        for (; c + NS <= A.full; c += kSlots) {
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int next = s + 1 < NS ? c + s + 1 : min(c + kSlots, A.full - 1);
#pragma unroll
                for (int i = 0; i < kKt; ++i) {
                    mul(s, i);
                    load(row, w, w_step, last, next, i, kl);
                }
            }
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            if (c + s >= A.chains) break;
#pragma unroll
            for (int i = 0; i < kKt; ++i) {
                weights(w, w_step, last, c + s, i);
#pragma unroll
                for (int m = 0; m < M; ++m)
                    x[i][m].load_end(row[m], ((c + s) * kKt + i) * 32 + kl, A.S.K);
                mul(s, i);
            }
        }
    }
};

// Few tokens: 16 of them, one rank tile and a part of the slots a workgroup, a wave a slot.
template <bool BF, bool I8>
__global__ __launch_bounds__(64 * kAdWaves) void k_shrink(AdArgs A) {
    __shared__ f32x4 part[kAdWaves][64];
    const moe_adapters& S = A.S;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // rank tiles, parts, pieces of tiles: those of a part of A side by side
    const int64_t item = by_xcd(blockIdx.x, A.items), piece = item % A.pieces;
    const int zr = (int)(item / A.pieces), z = zr % A.parts, r0 = zr / A.parts;
    const int64_t tile = A.sub > 1 ? piece / A.sub : piece;
    const int skip = A.sub > 1 ? (int)(piece % A.sub) * 16 : 0;
    const int32_t* rec = A.plan + tile * A.rec;
    const int a = rec[0], first = rec[1] + skip, count = rec[2] - skip;
    if (a >= S.n || count <= 0) return;
    const char* row[1] = {static_cast<const char*>(A.x) +
                          (int64_t)rec[4 + skip + (lane & 15)] * A.ldx * (I8 ? 1 : 2)};
    const uint8_t* w = static_cast<const uint8_t*>(S.a) +
                       (((int64_t)a * A.rt + r0) * A.kt * 64 + lane) * 16;
    Slots<BF, I8, 1, 1, 1> s;
    s.start(A, row, w, 0, 0, z * kAdWaves + wave, (lane >> 4) * 8);
    // the rank is looked at only now: the first loads are on their way
    if (r0 >= (S.ranks[a] + 15) / 16) return;
    s.run(A, row, w, 0, 0, z * kAdWaves + wave, (lane >> 4) * 8);
    part[wave][lane] = s.acc[0][0][0];
    __syncthreads();
    // lane l holds ranks (l >> 4) * 4 .. + 3 of token l & 15
    if (wave || (lane & 15) >= count) return;
    f32x4 v = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
    if constexpr (I8) v = v * A.x_scale[rec[4 + skip + (lane & 15)]];
    *reinterpret_cast<f32x4*>(A.h + (((int64_t)z * A.T + first + (lane & 15)) * A.rt + r0) * 16 +
                              (lane >> 4) * 4) = v * S.scales[a];
}

// fp16's power of two for a row of h, from the bits of its largest.
__device__ __forceinline__ int exponent_h(uint32_t most) { return (int)(most >> 23) - 127 - 14; }

// h (four ranks of a token) as the operand of the second product: two numbers each, in h3
// the third.  ex: fp16's power of two.
template <bool BF>
__device__ __forceinline__ u32x4 split_h(f32x4 v, int ex, uint2& h3) {
    float lo[4], lo3[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (BF) {
            // what would round past bf16's largest stays there, and the rest is in lo
            const float hi = __builtin_amdgcn_fmed3f(v[e], -0x1.fep127f, 0x1.fep127f);
            lo[e] = v[e] - (float)(__bf16)hi;
            lo3[e] = lo[e] - (float)(__bf16)lo[e];
            v[e] = hi;
        } else {
            v[e] = ldexpf(v[e], -ex);
            lo[e] = v[e] - (float)(_Float16)v[e];
        }
    }
    h3 = uint2{pack2<BF>(lo3[0], lo3[1]), pack2<BF>(lo3[2], lo3[3])};
    return u32x4{pack2<BF>(v[0], v[1]), pack2<BF>(v[2], v[3]), pack2<BF>(lo[0], lo[1]),
                 pack2<BF>(lo[2], lo[3])};
}

__device__ __forceinline__ uint32_t max_bits(f32x4 v) {
    uint32_t b = 0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) b = max(b, __float_as_uint(v[e]) & 0x7fffffffu);
    return b;
}

// Many tokens: 16 M of them and all the ranks a workgroup, two slots a wave.  h leaves it
// as the operand of the second product.
template <bool BF, bool I8, int M, int RTW>
__global__ __launch_bounds__(32 * kSlots, 2) void k_shrink_wide(AdArgs A) {
    constexpr int W = kSlots / 2;
    __shared__ f32x4 part[W][RTW * M][64];
    __shared__ uint32_t most[M * 16];
    const moe_adapters& S = A.S;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t piece = by_xcd(blockIdx.x, A.items), tile = piece / A.sub;
    const int skip = (int)(piece % A.sub) * 16 * M;
    const int32_t* rec = A.plan + tile * A.rec;
    const int a = rec[0], count = rec[2] - skip;
    if (a >= S.n || count <= 0) return;
    const char* row[M];
#pragma unroll
    for (int m = 0; m < M; ++m)
        row[m] = static_cast<const char*>(A.x) +
                 (int64_t)rec[4 + skip + 16 * m + (lane & 15)] * A.ldx * (I8 ? 1 : 2);
    const uint8_t* w = static_cast<const uint8_t*>(S.a) +
                       ((int64_t)a * A.rt * A.kt * 64 + lane) * 16;
    const int64_t w_step = (int64_t)A.kt * 1024;
    Slots<BF, I8, 2, M, RTW> s;
    s.start(A, row, w, w_step, A.rt - 1, 2 * wave, (lane >> 4) * 8);
    const int rts = min((S.ranks[a] + 15) / 16, A.rt);
    if (rts == 0) return;
    s.run(A, row, w, w_step, rts - 1, 2 * wave, (lane >> 4) * 8);
#pragma unroll
    for (int r = 0; r < RTW; ++r)
#pragma unroll
        for (int m = 0; m < M; ++m) part[wave][r * M + m][lane] = s.acc[0][r][m] + s.acc[1][r][m];
    if (tid < M * 16) most[tid] = 0u;
    __syncthreads();
    // four ranks of a token a thread
    constexpr int NO = (RTW * M * 64 + 32 * kSlots - 1) / (32 * kSlots);
    f32x4 v[NO];
    const float scale = S.scales[a];
#pragma unroll
    for (int i = 0; i < NO; ++i) {
        const int o = i * 32 * kSlots + tid, l = o & 63, m = (o >> 6) % M, r = (o >> 6) / M;
        const int t = 16 * m + (l & 15);
        if (r >= rts) continue;
        const f32x4* p = &part[0][0][0] + o;
        constexpr int N = RTW * M * 64;
        float xs = 1.f;
        if constexpr (I8) xs = A.x_scale[rec[4 + skip + t]];
        {
#pragma clang fp contract(off)
            // part by part and rounded, as k_shrink leaves them
            v[i] = (p[0] + p[N]) * xs * scale;
#pragma unroll
            for (int k = 2; k < W; k += 2)
                if (k / 2 < A.parts) v[i] = v[i] + (p[k * N] + p[(k + 1) * N]) * xs * scale;
        }
        if constexpr (!BF) atomicMax(&most[t], max_bits(v[i]));
    }
    if constexpr (!BF) __syncthreads();
#pragma unroll
    for (int i = 0; i < NO; ++i) {
        const int o = i * 32 * kSlots + tid, l = o & 63, m = (o >> 6) % M, r = (o >> 6) / M;
        if (r >= rts) continue;
        int ex = 0;
        if constexpr (!BF) {
            ex = exponent_h(most[16 * m + (l & 15)]);
            if (r == 0 && l < 16) A.hf[(piece * M + m) * 16 + l] = ldexpf(1.f, ex);
        }
        uint2 h3;
        const int64_t at = ((piece * M + m) * A.rt + r) * 64 + l;
        A.hh[at] = split_h<BF>(v[i], ex, h3);
        if (A.h3) A.h3[at] = h3;
    }
}

// ---------------------------------------------------------------- the second product

// Eight elements of y, of type YT, as loaded.
template <int YT>
struct RawY {
    u32x4 a, b;
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        constexpr int B = YT == MOE_DT_F32 ? 4 : 2;
        const char* q = static_cast<const char*>(p) + i * B;
        a = load16<false, true>(q);
        if constexpr (YT == MOE_DT_F32) b = load16<false, true>(q + 16);
    }
    __device__ __forceinline__ void f32(float (&v)[8]) const {
        if constexpr (YT == MOE_DT_F32) raw_to_f32(Raw8{a, b}, YT, v);
        else raw_to_f32(Raw8{a, a}, YT, v);
    }
};

// The weights of a group of 64 channels: row tiles 0 and 1 in b[r][0], 2 and 3 in b[r][1].
template <int RB>
struct Weights {
    u32x4 b[RB][2];
    __device__ __forceinline__ void load(const uint8_t* w, int last) {
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int p = 0; p < 2; ++p)
                b[r][p] = *reinterpret_cast<const u32x4*>(w + min(r, last) * 2048 + p * 1024);
    }
};

template <bool BF, bool THREE>
__device__ __forceinline__ void mul_h(const u32x4 (&b)[2], u32x4 hh, uint2 h3, f32x4 (&acc)[4]) {
    const uint2 hi = {hh[0], hh[1]}, lo = {hh[2], hh[3]};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint2 w = {b[j >> 1][(j & 1) * 2], b[j >> 1][(j & 1) * 2 + 1]};
        acc[j] = mma16<BF>(w, hi, acc[j]);
        acc[j] = mma16<BF>(w, lo, acc[j]);
        if constexpr (THREE) acc[j] = mma16<BF>(w, h3, acc[j]);
    }
}

// out = y + f * the products, 8 channels from n * 64 + g * 8 on and 8 from 32 after.
template <int YT>
__device__ __forceinline__ void finish(const AdArgs& A, int64_t token, int n, int g,
                                       const RawY<YT> (&y)[2], bool add, float f,
                                       const f32x4 (&acc)[4]) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float o[8];
        y[q].f32(o);
        if (add) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] += f * acc[2 * q + (e >> 2)][e & 3];
        }
        store_f32<8, false, true>(A.out, YT, token * A.ldo + n * 64 + q * 32 + g * 8, o);
    }
}

// The same where the group reaches past N.
template <int YT>
__device__ __forceinline__ void finish_end(const AdArgs& A, int64_t token, int n, int g, bool add,
                                           float f, const f32x4 (&acc)[4]) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = n * 64 + q * 32 + g * 8 + e;
            if (c >= A.S.N) continue;
            float one[1] = {load_elem(A.y, YT, token * A.ldy + c)};
            if (add) one[0] += f * acc[2 * q + (e >> 2)][e & 3];
            store_f32<1>(A.out, YT, token * A.ldo + c, one);
        }
}

// Few tokens: 16 a workgroup, whose waves share h and take the groups in turn.  RS: rank
// tiles of the set, at most.
template <bool BF, int YT, int RS>
__global__ __launch_bounds__(64 * kAdWaves, 2) void k_expand(AdArgs A) {
    constexpr bool THREE = BF && YT == MOE_DT_F32;
    constexpr int RB = RS < 8 ? RS : 8;          // rank tiles whose weights are in flight
    constexpr int NI = (RS + kAdWaves - 1) / kAdWaves;
    __shared__ u32x4 hs[RS][64];
    __shared__ uint2 hs3[THREE ? RS : 1][64];
    __shared__ uint32_t most[16];
    const moe_adapters& S = A.S;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t item = A.items0 + by_xcd(blockIdx.x, gridDim.x), piece = item % A.pieces;
    const int cg = (int)(item / A.pieces);
    const int64_t tile = A.sub > 1 ? piece / A.sub : piece;
    const int skip = A.sub > 1 ? (int)(piece % A.sub) * 16 : 0;
    const int32_t* rec = A.plan + tile * A.rec;
    const int a = rec[0], first = rec[1] + skip, count = rec[2] - skip;
    if (count <= 0) return;
    const bool mine = (lane & 15) < count;
    const int64_t token = rec[4 + skip + (lane & 15)];
    const int n = cg * A.per + wave, full = S.N / 64;
    RawY<YT> y[2];
    if (n < full) {
#pragma unroll
        for (int q = 0; q < 2; ++q) y[q].load(A.y, token * A.ldy + n * 64 + q * 32 + g * 8);
    }
    const int rts = a < S.n ? min((S.ranks[a] + 15) / 16, A.rt) : 0;
    if (rts == 0 && A.y == A.out) return;
    const uint8_t* w = static_cast<const uint8_t*>(S.b) +
                       ((int64_t)(rts ? a : 0) * A.groups + min(n, A.groups - 1)) * A.rt * 2048 +
                       lane * 16;
    Weights<RB> b;
    if (rts) b.load(w, rts - 1);

    // ------------------------------------------------ h: rank tile r is wave r % 4's
    float f = 1.f;
    f32x4 v[NI];
    const float* h = A.h + (int64_t)(first + min(lane & 15, count - 1)) * A.rt * 16 + g * 4;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int r = i * kAdWaves + wave;
        if (r >= rts) continue;
        f32x4 p[kAdParts];
#pragma unroll
        for (int z = 0; z < kAdParts; ++z)
            if (z < A.parts) p[z] = *reinterpret_cast<const f32x4*>(h + z * A.T * A.rt * 16 + r * 16);
        v[i] = p[0];
#pragma unroll
        for (int z = 1; z < kAdParts; ++z)
            if (z < A.parts) v[i] = v[i] + p[z];
    }
    int ex = 0;
    if constexpr (!BF) {
        if (tid < 16) most[tid] = 0u;
        __syncthreads();
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < NI; ++i) m = max(m, max_bits(v[i]));
        atomicMax(&most[lane & 15], m);
        __syncthreads();
        ex = exponent_h(most[lane & 15]);
        f = ldexpf(1.f, ex);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int r = i * kAdWaves + wave;
        if (r >= rts) continue;
        uint2 h3;
        hs[r][lane] = split_h<BF>(v[i], ex, h3);
        if constexpr (THREE) hs3[r][lane] = h3;
    }
    __syncthreads();
    if (n >= A.groups) return;

    // ------------------------------------------------ the products
    f32x4 acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r0 = 0; r0 < RS; r0 += RB) {
        if (r0 >= rts) break;
        if (r0) b.load(w + r0 * 2048, rts - 1 - r0);
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            if (r0 + r >= rts) break;
            mul_h<BF, THREE>(b.b[r], hs[r0 + r][lane], hs3[THREE ? r0 + r : 0][lane], acc);
        }
    }
    if (!mine) return;
    if (n < full) finish<YT>(A, token, n, g, y, rts > 0, f, acc);
    else finish_end<YT>(A, token, n, g, rts > 0, f, acc);
}

// Many tokens: 16 M and `per` groups a wave; the waves of a workgroup neighbouring tokens,
// which as a rule share their adapter and so its weights in the L1.
template <bool BF, int YT, int M, int RS>
__global__ __launch_bounds__(64 * kAdWaves) void k_apply(AdArgs A) {
    constexpr bool THREE = BF && YT == MOE_DT_F32;
    const moe_adapters& S = A.S;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int64_t item = A.items0 + by_xcd(blockIdx.x, gridDim.x);
    const int64_t piece = item % A.pieces * kAdWaves +
                          __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cg = (int)(item / A.pieces);
    if (piece >= A.tiles * A.sub) return;
    const int skip = (int)(piece % A.sub) * 16 * M;
    const int32_t* rec = A.plan + piece / A.sub * A.rec;
    const int a = rec[0], count = rec[2] - skip;
    if (count <= 0) return;
    int64_t token[M];
#pragma unroll
    for (int m = 0; m < M; ++m) token[m] = rec[4 + skip + 16 * m + (lane & 15)];
    const int n0 = cg * A.per, n1 = min(n0 + A.per, A.groups), full = min(n1, S.N / 64);
    RawY<YT> next[M][2];
    auto load_y = [&](int n) {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                next[m][q].load(A.y, token[m] * A.ldy + n * 64 + q * 32 + g * 8);
    };
    if (n0 < full) load_y(n0);
    const int rts = a < S.n ? min((S.ranks[a] + 15) / 16, A.rt) : 0;
    if (rts == 0 && A.y == A.out) return;
    u32x4 hh[M][RS];
    uint2 h3[M][THREE ? RS : 1];
    float f[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int64_t p = piece * M + m;
        f[m] = 1.f;
        if constexpr (!BF)
            if (rts) f[m] = A.hf[p * 16 + (lane & 15)];
#pragma unroll
        for (int r = 0; r < RS; ++r) {
            if (r < rts) hh[m][r] = A.hh[(p * A.rt + r) * 64 + lane];
            if constexpr (THREE)
                if (r < rts) h3[m][r] = A.h3[(p * A.rt + r) * 64 + lane];
        }
    }
    const uint8_t* w = static_cast<const uint8_t*>(S.b) +
                       (int64_t)(rts ? a : 0) * A.groups * A.rt * 2048 + lane * 16;
    Weights<RS> b;
    f32x4 acc[4];
    auto products = [&](int m) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < RS; ++r) {
            if (r >= rts) break;
            mul_h<BF, THREE>(b.b[r], hh[m][r], h3[m][THREE ? r : 0], acc);
        }
    };
    int n = n0;
    for (; n < full; ++n) {
        if (rts) b.load(w + (int64_t)n * A.rt * 2048, rts - 1);
        RawY<YT> y[M][2];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int q = 0; q < 2; ++q) y[m][q] = next[m][q];
        if (n + 1 < full) load_y(n + 1);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            products(m);
            if (16 * m + (lane & 15) < count) finish<YT>(A, token[m], n, g, y[m], rts > 0, f[m], acc);
        }
    }
    if (n < n1) {
        if (rts) b.load(w + (int64_t)n * A.rt * 2048, rts - 1);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            products(m);
            if (16 * m + (lane & 15) < count) finish_end<YT>(A, token[m], n, g, rts > 0, f[m], acc);
        }
    }
}

// 16 bytes of a slot's tiles a thread: A's first, then B's.
__global__ __launch_bounds__(256) void k_pack(moe_adapters S, int slot, const uint16_t* a,
                                              int64_t lda, const uint16_t* b, int64_t ldb, int rank,
                                              float scale, int rt, int kt, int64_t na, int64_t nb) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i == 0) {
        const_cast<int32_t*>(S.ranks)[slot] = rank;
        const_cast<float*>(S.scales)[slot] = scale;
    }
    u32x4 v = {0u, 0u, 0u, 0u};
    if (i < na) {
        const int l = (int)(i & 63);
        const int64_t tile = i >> 6;
        const int r = (int)(tile / kt) * 16 + (l & 15);
        const int k = (int)(tile % kt) * 32 + (l >> 4) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (r < rank && k + e < S.K) v[e >> 1] |= (uint32_t)a[r * lda + k + e] << (16 * (e & 1));
        reinterpret_cast<u32x4*>(const_cast<void*>(S.a))[slot * na + i] = v;
    } else if (i < na + nb) {
        const int64_t q = i - na;
        const int l = (int)(q & 63), p = (int)(q >> 6) & 1;
        const int64_t tile = q >> 7;
        const int row = l & 15, r = (int)(tile % rt) * 16 + (l >> 4) * 4;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t n = tile / rt * 64 + p * 32 + (row >> 2) * 8 + (e >> 2) * 4 + (row & 3);
            const int k = r + (e & 3);
            if (n < S.N && k < rank) v[e >> 1] |= (uint32_t)b[n * ldb + k] << (16 * (e & 1));
        }
        reinterpret_cast<u32x4*>(const_cast<void*>(S.b))[slot * nb + q] = v;
    }
}

// The kernels for many tokens read x and the weights once for all of an adapter's ranks
// and 32 tokens, the others once for each 16; but fewer workgroups hold less in flight.
// Ranks 17 to 128 from T times rank tiles 8192 on, whatever the widths (8 adapters, us
// against the others, for 6144 -> 6144, 6144 -> 1024, 1024 -> 6144, 256 -> 6144, 6144 -> 256):
//   rank 32, 2800 tokens   46.0 : 44.4   23.8 : 23.3   21.7 : 25.1   20.0 : 20.7   23.1 : 21.0
//   rank 32, 4096          55.0 : 64.8   25.9 : 31.6   36.9 : 43.0   34.9 : 37.1   23.4 : 28.4
//   rank 64, 1500          34.0 : 36.8   27.9 : 27.3   19.2 : 21.7   17.3 : 17.2   27.3 : 25.9
//   rank 64, 2048          38.3 : 45.8   28.2 : 31.7   22.6 : 26.2   20.9 : 20.6   27.3 : 29.2
//   rank 128, 1024         40.1 : 43.7   31.8 : 33.3   22.7 : 25.7   19.7 : 19.2   31.5 : 31.7
// Rank 16 stays with the others (4096 tokens, 6144 -> 6144: 51.6 : 47.4); past 128 there are
// none for many tokens (rank 256: 258 us, against 111 of rank 128).
bool ad_wide(const moe_adapters& S, int64_t T) {
    const int64_t rt = ad_rank_tiles(S.rank);
    return ad_plan(T, S.n).tile == 64 && rt >= 2 && rt <= kWideTiles && T * rt >= 8192;
}

}  // namespace

// h: fp32 parts, or (many tokens) 24 bytes for four ranks of a token and 4 a token; the
// larger, so that a workspace serves fewer tokens too.
size_t add_adapters_ws_bytes(const moe_adapters& S, int64_t T) {
    const AdPlan lay = ad_plan(T, S.n);
    const size_t rt = (size_t)ad_rank_tiles(S.rank);
    const size_t pieces = (size_t)(lay.tiles * (lay.tile / 16));
    const size_t few = (size_t)T * rt * 64 * ad_parts(S.K);
    const size_t many = ad_wide(S, T) ? pieces * (rt * 64 * 24 + 64) : 0;
    return few > many ? few : many;
}

int launch_pack_adapter(const moe_adapters& S, int32_t slot, const void* a, int64_t lda,
                        const void* b, int64_t ldb, int32_t rank, float scale, void* stream) {
    const int rt = (int)ad_rank_tiles(S.rank), kt = (int)ad_chains(S.K) * kKt;
    // a slot that is emptied keeps its bytes: no call reads them
    const int64_t na = rank ? ad_a_bytes(S.rank, S.K) / 16 : 0;
    const int64_t nb = rank ? ad_b_bytes(S.rank, S.N) / 16 : 0;
    k_pack<<<(unsigned)((na + nb + 256) / 256), 256, 0, reinterpret_cast<hipStream_t>(stream)>>>(
        S, slot, static_cast<const uint16_t*>(a), lda, static_cast<const uint16_t*>(b), ldb, rank,
        scale, rt, kt, na, nb);
    MOEQ_CHECK_LAUNCH();
    return MOE_OK;
}

int launch_add_adapters(const moe_adapters& S, const void* x, int32_t x_dtype, int64_t ldx,
                        const float* x_scale, const int32_t* plan, int64_t T, const void* y,
                        void* out, int32_t y_dtype, int64_t ldy, int64_t ldo, float* h,
                        void* stream) {
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const AdPlan lay = ad_plan(T, S.n);
    AdArgs A{};
    A.S = S;
    A.x = x;
    A.ldx = ldx;
    A.x_scale = x_scale;
    A.plan = plan;
    A.h = h;
    A.y = y;
    A.out = out;
    A.ldy = ldy;
    A.ldo = ldo;
    A.T = T;
    A.tiles = lay.tiles;
    A.rec = lay.rec;
    A.rt = (int)ad_rank_tiles(S.rank);
    A.chains = (int)ad_chains(S.K);
    A.kt = A.chains * kKt;
    A.full = (int)((x_dtype == MOE_DT_I8 ? round_up(S.K, kI8TileK) : S.K) / kAdChain);
    A.parts = ad_parts(S.K);
    A.groups = (S.N + 63) / 64;
    const bool wide = ad_wide(S, T);
    if (wide) {
        const int64_t n = lay.tiles * (lay.tile / 16);
        A.hh = reinterpret_cast<u32x4*>(h);
        A.h3 = reinterpret_cast<uint2*>(A.hh + n * A.rt * 64);
        A.hf = reinterpret_cast<float*>(A.h3 + n * A.rt * 64);
        if (y_dtype != MOE_DT_F32 || S.w_dtype != MOE_DT_BF16) A.h3 = nullptr;
    }
    using std::integral_constant;
    integral_constant<int, 1> c1;
    integral_constant<int, 2> c2;
    integral_constant<int, 4> c4;
    integral_constant<int, 8> c8;
    integral_constant<int, 16> c16;
    auto shrink = [&](auto bf, auto i8) {
        constexpr bool BF = decltype(bf)::value, I8 = decltype(i8)::value;
        auto go = [&](auto m, auto rtw) {
            constexpr int M = decltype(m)::value, RTW = decltype(rtw)::value;
            A.sub = lay.tile / 16 / M;
            A.items = lay.tiles * A.sub;
            k_shrink_wide<BF, I8, M, RTW><<<(unsigned)A.items, 32 * kSlots, 0, s>>>(A);
        };
        if (!wide) {
            A.sub = lay.tile / 16;
            A.pieces = lay.tiles * A.sub;
            A.items = A.pieces * A.rt * A.parts;
            k_shrink<BF, I8><<<(unsigned)A.items, 64 * kAdWaves, 0, s>>>(A);
        } else if (A.rt == 2) {
            go(c2, c2);
        } else if (A.rt <= 4) {
            go(c2, c4);
        } else {
            go(c1, c8);
        }
    };
    auto expand = [&](auto bf, auto rs) {
        constexpr bool BF = decltype(bf)::value;
        constexpr int RS = decltype(rs)::value;
        constexpr int M = RS <= 4 ? 2 : 1;
        const int64_t max_items = rows_of_launch(kAdWaves);
        A.sub = wide ? lay.tile / 16 / M : lay.tile / 16;
        A.pieces = lay.tiles * A.sub;
        if (wide) A.pieces = (A.pieces + kAdWaves - 1) / kAdWaves;
        A.per = wide ? 2 : kAdWaves;
        A.cgs = (A.groups + A.per - 1) / A.per;
        A.items = A.pieces * A.cgs;
        for (A.items0 = 0; A.items0 < A.items; A.items0 += max_items) {
            const int64_t n = A.items - A.items0 < max_items ? A.items - A.items0 : max_items;
            auto go = [&](auto yt) {
                constexpr int YT = decltype(yt)::value;
                if constexpr (RS > 1 && RS <= kWideTiles) {
                    if (wide) {
                        k_apply<BF, YT, M, RS><<<(unsigned)n, 64 * kAdWaves, 0, s>>>(A);
                        return;
                    }
                }
                k_expand<BF, YT, RS><<<(unsigned)n, 64 * kAdWaves, 0, s>>>(A);
            };
            if (y_dtype == MOE_DT_F32) go(integral_constant<int, MOE_DT_F32>{});
            else if (y_dtype == MOE_DT_BF16) go(integral_constant<int, MOE_DT_BF16>{});
            else go(integral_constant<int, MOE_DT_F16>{});
        }
    };
    auto run = [&](auto bf) {
        if (x_dtype == MOE_DT_I8) shrink(bf, std::true_type{});
        else shrink(bf, std::false_type{});
        if (A.rt == 1) expand(bf, c1);
        else if (A.rt == 2) expand(bf, c2);
        else if (A.rt <= 4) expand(bf, c4);
        else if (A.rt <= 8) expand(bf, c8);
        else expand(bf, c16);
    };
    if (S.w_dtype == MOE_DT_BF16) run(std::true_type{});
    else run(std::false_type{});
    MOEQ_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace moeq
