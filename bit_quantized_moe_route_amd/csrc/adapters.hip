// Low-rank adapters of many requests beside a projection that they share:
//
//   h[t] = s_a * x_scale[t] * A_a x[t]           (rank r_a, fp32)
//   out[t] = y[t] + B_a h[t]                     (one rounding to y's type)
//
// a the adapter of token t's request.  Tokens go in tiles of up to 16 of one adapter
// (the plan of a batch); two launches, so that both products spread over the chip:
// the shrink gives a workgroup a tile and some of its rank tiles, its 16 waves the
// inputs (chains of 128, wave w those of w, w + 16, ...), joined in LDS in wave order;
// the expand gives a wave a tile and groups of 64 channels.  A token's bits depend on
// nothing but its row and its adapter.
//
// Both products are matrix instructions of 16 x 16 x 32 on 16-bit operands with fp32
// sums.  x and the weights are 16-bit as they are (8-bit codes are exact in either
// type).  h stays fp32-like in the expand: it enters as the sum of two numbers of the
// weights' type, both in one instruction (the inner 32 are 16 ranks of the first and
// the same 16 of the second, against the same weights twice).  fp16 holds 22 bits of h
// so, its row first brought to [1, 2) by a power of two; bf16 16 bits, enough for a
// 16-bit result, and a third number follows where y is fp32.
#include <type_traits>

#include "elem_dev.h"

namespace moeq {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kShrinkWaves = 16;
constexpr int kKt = kAdChain / 32;              // input tiles of a chain

struct AdArgs {
    moe_adapters S;
    const void* x;
    int64_t ldx;
    const float* x_scale;
    const int32_t* plan;
    int64_t order, tiles;       // places in the plan
    float* h;                   // [T][rt * 16]
    const void* y;
    void* out;
    int64_t ldy, ldo;
    int64_t max_tiles, task0, tasks;
    int y_dtype;
    int rt, kt, groups;         // rank tiles, input tiles, groups of 64 channels
    int per, cgs;               // expand: groups of a wave, such pieces of a row
    bool tile_fast;
};

// D += A * B over a 16 x 16 x 32 tile; operands as eight 16-bit values a lane.
template <bool BF>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 acc) {
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
    else
        return mfma16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), acc);
}

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return BF ? pack_bf16(lo, hi) : pack_f16(lo, hi);
}

// Eight inputs of a row from k on, as the weights' type; past K zeros.
template <bool BF, bool I8>
__device__ __forceinline__ u32x4 load_x(const void* row, int k, int K) {
    if constexpr (I8) {
        u32x4 r = {0u, 0u, 0u, 0u};
        if (k < K) {             // rows are padded with zero codes to 64
            const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const int8_t*>(row) + k);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t w = p < 2 ? q.x : q.y;
                const int sh = (p & 1) * 16;
                r[p] = pack2<BF>((float)(int8_t)(w >> sh), (float)(int8_t)(w >> (sh + 8)));
            }
        }
        return r;
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(row);
        if (k + 8 <= K) return load16<false, true>(p + k);
        u32x4 r = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < K) r[e >> 1] |= (uint32_t)p[k + e] << (16 * (e & 1));
        return r;
    }
}

template <bool BF, bool I8, int RTW>
__global__ __launch_bounds__(64 * kShrinkWaves) void k_shrink(AdArgs A) {
    __shared__ f32x4 part[kShrinkWaves][RTW][64];
    const moe_adapters& S = A.S;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if ((int)blockIdx.x >= A.plan[0]) return;
    const int32_t* tile = A.plan + A.tiles + 4 * (int64_t)blockIdx.x;
    const int a = tile[0], first = tile[1], count = tile[2];
    if (a >= S.n) return;
    const int rts = min((S.ranks[a] + 15) / 16, A.rt);
    const int r0 = blockIdx.y * RTW;
    if (r0 >= rts) return;
    const int pos = first + min(lane & 15, count - 1);
    const int64_t token = A.plan[A.order + pos];
    const char* row = static_cast<const char*>(A.x) + token * A.ldx * (I8 ? 1 : 2);
    const uint8_t* w = static_cast<const uint8_t*>(S.a) +
                       (((int64_t)a * A.rt + r0) * A.kt * 64 + lane) * 16;
    const int64_t w_step = (int64_t)A.kt * 1024;
    const int chains = A.kt / kKt;

    f32x4 acc[RTW];
#pragma unroll
    for (int r = 0; r < RTW; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int kl = (lane >> 4) * 8;
    u32x4 xn[kKt];
#pragma unroll
    for (int i = 0; i < kKt; ++i)
        xn[i] = load_x<BF, I8>(row, (wave * kKt + i) * 32 + kl, wave < chains ? S.K : 0);
    for (int c = wave; c < chains; c += kShrinkWaves) {
        u32x4 x[kKt], wt[RTW][kKt];
#pragma unroll
        for (int r = 0; r < RTW; ++r)
#pragma unroll
            for (int i = 0; i < kKt; ++i)
                // past the adapter's own ranks: the last tile again, whose sums are dropped
                wt[r][i] = *reinterpret_cast<const u32x4*>(
                    w + min(r, rts - 1 - r0) * w_step + ((int64_t)c * kKt + i) * 1024);
        const int nc = c + kShrinkWaves;
#pragma unroll
        for (int i = 0; i < kKt; ++i) {
            x[i] = xn[i];
            xn[i] = load_x<BF, I8>(row, (nc * kKt + i) * 32 + kl, nc < chains ? S.K : 0);
        }
#pragma unroll
        for (int i = 0; i < kKt; ++i)
#pragma unroll
            for (int r = 0; r < RTW; ++r) acc[r] = mma<BF>(wt[r][i], x[i], acc[r]);
    }
#pragma unroll
    for (int r = 0; r < RTW; ++r) part[wave][r][lane] = acc[r];
    __syncthreads();
    const float* p = reinterpret_cast<const float*>(part);
    const int o = tid;                           // rank tile, lane and rank of a result
    if (o >= RTW * 256) return;
    const int r = o >> 8, l = (o >> 2) & 63;
    if (r0 + r >= rts || (l & 15) >= count) return;
    float s = p[o];
    const int parts = min(kShrinkWaves, chains);
    for (int i = 1; i < parts; ++i) s += p[i * RTW * 256 + o];
    if constexpr (I8) s *= A.x_scale[A.plan[A.order + first + (l & 15)]];
    A.h[(int64_t)(first + (l & 15)) * A.rt * 16 + (r0 + r) * 16 + (l >> 4) * 4 + (o & 3)] =
        s * S.scales[a];
}

// RS: rank tiles of the set, at most.
template <bool BF, int RS>
__global__ __launch_bounds__(256) void k_expand(AdArgs A) {
    constexpr int RB = RS < 4 ? RS : 4;          // rank tiles whose weights are in flight
    const moe_adapters& S = A.S;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int64_t task = A.task0 + (int64_t)blockIdx.x * 4 +
                         __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (task >= A.tasks) return;
    const int64_t t = A.tile_fast ? task % A.max_tiles : task / A.cgs;
    const int cg = (int)(A.tile_fast ? task / A.max_tiles : task % A.cgs);
    if (t >= A.plan[0]) return;
    const int32_t* tile = A.plan + A.tiles + 4 * t;
    const int a = tile[0], first = tile[1], count = tile[2];
    const int rts = a < S.n ? min((S.ranks[a] + 15) / 16, A.rt) : 0;
    if (rts == 0 && A.y == A.out) return;
    const bool mine = (lane & 15) < count;
    const int pos = first + min(lane & 15, count - 1);
    const int64_t token = A.plan[A.order + pos];
    const int yt = A.y_dtype;
    const int64_t yrow = token * A.ldy, orow = token * A.ldo;
    const bool third = BF && yt == MOE_DT_F32;

    // ------------------------------------------------ h as two (three) 16-bit numbers
    u32x4 hh[RS], h3[BF ? RS : 1];
    float f = 1.f;
    {
        const float* h = A.h + (int64_t)pos * A.rt * 16 + (g & 1) * 8;
        f32x4 v[RS][2];
#pragma unroll
        for (int r = 0; r < RS; ++r) {
            if (r < rts) {
                v[r][0] = *reinterpret_cast<const f32x4*>(h + r * 16);
                v[r][1] = *reinterpret_cast<const f32x4*>(h + r * 16 + 4);
            } else {
                v[r][0] = v[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
        }
        int ex = 0;
        if constexpr (!BF) {
            float m = 0.f;
#pragma unroll
            for (int r = 0; r < RS; ++r)
#pragma unroll
                for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[r][e >> 2][e & 3]));
            m = fmaxf(m, __shfl_xor(m, 16));
            ex = (int)(__float_as_uint(m) >> 23) - 127;
            f = ldexpf(1.f, ex);
        }
#pragma unroll
        for (int r = 0; r < RS; ++r) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float p[2], lo[2], lo3[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    p[e] = v[r][q >> 1][(q & 1) * 2 + e];
                    if constexpr (!BF) p[e] = ldexpf(p[e], -ex);
                    if constexpr (BF) {
                        lo[e] = p[e] - (float)(__bf16)p[e];
                        lo3[e] = lo[e] - (float)(__bf16)lo[e];
                    } else {
                        lo[e] = p[e] - (float)(_Float16)p[e];
                    }
                }
                hh[r][q] = g < 2 ? pack2<BF>(p[0], p[1]) : pack2<BF>(lo[0], lo[1]);
                if constexpr (BF) h3[r][q] = g < 2 ? pack_bf16(lo3[0], lo3[1]) : 0u;
            }
        }
    }

    const uint8_t* w = static_cast<const uint8_t*>(S.b) +
                       (int64_t)(rts ? a : 0) * A.groups * A.rt * 2048 + (lane & 31) * 16;
    const int n0 = cg * A.per, n1 = min(n0 + A.per, A.groups);
    for (int n = n0; n < n1; ++n) {
        // this lane's two runs of 8 channels
        int ch[2];
        Raw8 y[2];
        bool whole[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            ch[q] = n * 64 + q * 32 + g * 8;
            whole[q] = ch[q] + 8 <= S.N;
            if (mine && whole[q]) y[q] = load_raw8<false, true>(A.y, yt, yrow + ch[q]);
        }
        f32x4 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        const uint8_t* wn = w + (int64_t)n * A.rt * 2048;
#pragma unroll
        for (int r0 = 0; r0 < RS; r0 += RB) {
            if (r0 >= rts) break;
            u32x4 b[RB][4];
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    b[r][j] = *reinterpret_cast<const u32x4*>(
                        wn + min(r0 + r, rts - 1) * 2048 + j * 512);
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                if (r0 + r >= rts) break;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[j] = mma<BF>(b[r][j], hh[r0 + r], acc[j]);
                    if constexpr (BF)
                        if (third) acc[j] = mma<BF>(b[r][j], h3[r0 + r], acc[j]);
                }
            }
        }
        if (!mine) continue;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = f * acc[2 * q + (e >> 2)][e & 3];
            if (whole[q]) {
                float o[8];
                raw_to_f32(y[q], yt, o);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = rts ? o[e] + v[e] : o[e];
                store_f32<8, false, true>(A.out, yt, orow + ch[q], o);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (ch[q] + e >= S.N) continue;
                    const float o = load_elem(A.y, yt, yrow + ch[q] + e);
                    const float one[1] = {rts ? o + v[e] : o};
                    store_f32<1>(A.out, yt, orow + ch[q] + e, one);
                }
            }
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
        const int l = (int)(q & 31), j = (int)(q >> 5) & 3;
        const int64_t tile = q >> 7;
        const int row = l & 15;
        const int64_t n = tile / rt * 64 + (j >> 1) * 32 + (row >> 2) * 8 + (j & 1) * 4 + (row & 3);
        const int r = (int)(tile % rt) * 16 + (l >> 4) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (n < S.N && r + e < rank) v[e >> 1] |= (uint32_t)b[n * ldb + r + e] << (16 * (e & 1));
        reinterpret_cast<u32x4*>(const_cast<void*>(S.b))[slot * nb + q] = v;
    }
}

}  // namespace

int launch_pack_adapter(const moe_adapters& S, int32_t slot, const void* a, int64_t lda,
                        const void* b, int64_t ldb, int32_t rank, float scale, void* stream) {
    const int rt = (int)ad_rank_tiles(S.rank), kt = (int)(ad_a_bytes(16, S.K) / 1024);
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
    A.order = lay.order;
    A.tiles = lay.tiles;
    A.h = h;
    A.y = y;
    A.out = out;
    A.ldy = ldy;
    A.ldo = ldo;
    A.max_tiles = lay.max_tiles;
    A.y_dtype = y_dtype;
    A.rt = (int)ad_rank_tiles(S.rank);
    A.kt = (int)(ad_a_bytes(16, S.K) / 1024);
    A.groups = (S.N + 63) / 64;

    const bool many = T >= 1024;
    auto shrink = [&](auto bf, auto i8, auto rtw) {
        constexpr int RTW = decltype(rtw)::value;
        k_shrink<decltype(bf)::value, decltype(i8)::value, RTW>
            <<<dim3((unsigned)A.max_tiles, (unsigned)((A.rt + RTW - 1) / RTW)), 64 * kShrinkWaves, 0,
               s>>>(A);
    };
    A.tile_fast = many;
    A.per = many ? 8 : 1;
    A.cgs = (A.groups + A.per - 1) / A.per;
    A.tasks = A.max_tiles * A.cgs;
    auto expand = [&](auto bf, auto rs) {
        const int64_t most = rows_of_launch(4) * 4;
        for (A.task0 = 0; A.task0 < A.tasks; A.task0 += most) {
            const int64_t n = A.tasks - A.task0 < most ? A.tasks - A.task0 : most;
            k_expand<decltype(bf)::value, decltype(rs)::value>
                <<<(unsigned)((n + 3) / 4), 256, 0, s>>>(A);
        }
    };
    std::integral_constant<int, 1> c1;
    std::integral_constant<int, 2> c2;
    std::integral_constant<int, 4> c4;
    std::integral_constant<int, 8> c8;
    std::integral_constant<int, 16> c16;
    auto run = [&](auto bf) {
        auto by = [&](auto rtw) {
            if (x_dtype == MOE_DT_I8) shrink(bf, std::true_type{}, rtw);
            else shrink(bf, std::false_type{}, rtw);
        };
        if (!many || A.rt == 1) by(c1);
        else if (A.rt == 2) by(c2);
        else by(c4);
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
