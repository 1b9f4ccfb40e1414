// Products in 8-bit integers for many rows: a grouped GEMM on
// v_mfma_i32_32x32x32_i8 with the same results, bit for bit, as the
// weight-streaming kernels (the sums are exact).
//
// A workgroup of 4 waves owns BM token rows of one expert (or of the whole
// batch) x 256 record rows; each wave 64 of them: two 32-channel tiles, or 32
// gate and the matching 32 up channels, so that SwiGLU is done in registers.
//   * weights go straight from the packed tiles to registers (each byte is
//     read by one wave), the next 128 inputs in flight while the current are
//     multiplied;
//   * the BM x 128 token codes are gathered through registers into LDS,
//     double-buffered, 16-byte chunks XOR-swizzled by row.  (Direct-to-LDS loads
//     make the compiler wait for all of them before any LDS read: 229 us against
//     184 for the case below.)
//
// What bounds it: the matrix cores for one large matrix (4096 tokens, 6144 x
// 6144: 144 to 150 us, 2.06 to 2.15 POP/s; the library's 8192^3 product reached
// 2.03 on the same card); the weights' stream for routed experts, whose bytes
// are read once a tile (8 of 256, H 6144, I 2048: 1.74 ms at 1024 tokens, 1.82
// at 2048, 2.26 at 4096: 1.44 gate/up, 0.055 codes of h, 0.74 down.  The gate/up
// pass there fetches 8.0 GB for 6.4 GB of weights, since half of the experts
// have over 128 rows and their second tile finds two thirds of its weights in
// L2; without its 268 MB of h stores it would take 1.22 ms, without its products
// no less.  Tiles of 64 or 96 rows, two tiles in one workgroup, blocked weight
// layouts and two stages in flight were all slower or no faster); the weights'
// loads of one workgroup per CU in between (500 tokens, 6144 x 6144: 40 us, 26
// without them; 8 waves a workgroup, 3 or 4 stages in flight, another first input
// for each workgroup: no faster).
#include <type_traits>

#include "i8_dev.h"

namespace moeq {

namespace {

typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

constexpr int kStageK = 128;

__device__ __forceinline__ i32x16 mfma_i8_32(u32x4 a, u32x4 b, i32x16 acc) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), acc, 0, 0, 0);
}

struct GemmTile {
    int e, n;            // expert (-1: none), channel tile
    int64_t r0;          // first row
    int rows;            // at most BM
};

// Workgroup blk's tile.  The list of tiles goes by expert, channel tile and
// token tile (fastest); workgroups are dealt to the XCDs round-robin by the
// hardware, and XCD x takes positions [kRun x, kRun (x + 1)) of every 8 kRun,
// so that neighbours, which share weights or tokens, run beside each other on
// one L2.
constexpr int kRun = 8;

template <int BM>
__device__ __forceinline__ GemmTile find_tile(const I8Pass& A, int blk, int nnt, int lane) {
    GemmTile g{-1, 0, 0, 0};
    const int pos = ((blk >> 3) / kRun * 8 + (blk & 7)) * kRun + (blk >> 3) % kRun;
    // the i-th of nm tiles over m rows, all of nearly the same number
    auto cut = [&](int64_t r0, int64_t m, int nm, int i) {
        const int64_t per = (m + nm - 1) / nm;
        g.r0 = r0 + i * per;
        g.rows = (int)max((int64_t)0, min(per, m - i * per));
    };
    if (!A.offsets) {
        const int nm = (int)((A.T + BM - 1) / BM);
        if (pos / nm >= nnt) return g;
        g.e = 0;
        g.n = pos / nm;
        cut(0, A.T, nm, pos % nm);
        return g;
    }
    const int want = pos / nnt;
    int before = 0;
    for (int e0 = 0; e0 < A.E; e0 += 256) {
        const Offsets4 o = load_offsets(A.offsets, A.E, e0, lane);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int nm = (o.o1[c] - o.o0[c] + BM - 1) / BM;
            int incl = nm;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int v = __shfl_up(incl, off);
                if (lane >= off) incl += v;
            }
            const int tot = __builtin_amdgcn_readlane(incl, 63);
            if (want < before + tot) {
                const int w = want - before;
                const uint64_t mask = __ballot(w >= incl - nm && w < incl);
                const int owner = uniform(__ffsll((unsigned long long)mask) - 1);
                const int nmo = __builtin_amdgcn_readlane(nm, owner);
                const int r = pos - (before + __builtin_amdgcn_readlane(incl, owner) - nmo) * nnt;
                const int a = __builtin_amdgcn_readlane(o.o0[c], owner);
                g.e = e0 + 64 * c + owner;
                g.n = r / nmo;
                cut(a, __builtin_amdgcn_readlane(o.o1[c], owner) - a, nmo, r % nmo);
                return g;
            }
            before += tot;
        }
    }
    return g;
}

// CW waves side by side over the channels, 64 each; KP sets of them split the
// inputs and add their int32 sums in LDS.
template <bool PAIR, int BM, int CW, int KP>
__global__ __launch_bounds__(64 * CW * KP, 2) void k_gemm_i8(I8Pass A, int ngroups, int nnt,
                                                             bool pairs) {
    constexpr int NT = BM / 32;                  // 32-row token tiles
    constexpr int XW = 4 / CW;                   // token loads of a wave per 32 rows
    __shared__ __attribute__((aligned(1024))) uint8_t tokens[KP][2][BM * kStageK];
    __shared__ int32_t sums[KP > 1 ? BM * 64 * CW : 1];
    __shared__ float qs[BM];
    const int lane = threadIdx.x & 63, wave = uniform((threadIdx.x >> 6) % CW);
    const int part = uniform((threadIdx.x >> 6) / CW);
    auto& tok = tokens[part];
    const GemmTile t = find_tile<BM>(A, blockIdx.x, nnt, lane);
    if (t.e < 0 || t.rows == 0) return;
    const int Kp = (A.K + kI8TileK - 1) / kI8TileK * kI8TileK;
    const int ns = (A.K + kStageK - 1) / kStageK;
    // this part's stages, and those of the longest part
    const int sa = ns * part / KP, se = ns * (part + 1) / KP, steps = (ns + KP - 1) / KP;
    const int left = t.rows;
    const int64_t first = t.r0;
    auto source = [&](int row) -> int64_t {
        const int64_t r = first + min(row, left - 1);
        return A.offsets && A.perm_src ? A.perm_src[r] / A.k : r;
    };
    if ((int)threadIdx.x < BM) qs[threadIdx.x] = A.qscale[source(threadIdx.x)];

    // tokens: load (i, h) of a wave covers rows 32 i + 8 (wave XW + h) .. + 8
    const int8_t* xp[NT][XW];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int h = 0; h < XW; ++h)
            xp[i][h] = A.q + source(32 * i + 8 * (wave * XW + h) + (lane >> 3)) * A.ldq;
    // chunk c of row r lies at chunk c ^ (r & 7): reads of 8 rows hit all banks
    const int xat = (wave * XW * 8 + (lane >> 3)) * kStageK + ((lane & 7) ^ (lane >> 3)) * 16;

    // weights: tiles c = 0, 1 of this wave's 64 record rows; a lane's column is
    // channel lane & 31 of the gate (0) and up (1) rows, or, one matrix alone,
    // record row 2 (lane & 31) + c, so that a lane has two neighbours to store.
    const int g0 = (t.n * CW + wave) * 4;
    const int col = lane & 31;
    const uint8_t* wp[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int r = PAIR ? col : 2 * col + c;
        const int g = min(g0 + (PAIR ? 2 * (r >> 4) + c : r >> 4), ngroups - 1);
        wp[c] = A.w + t.e * A.w_stride + (int64_t)g * (2 * ns) * kI8TileBytes + (lane >> 5) * 256 +
                (r & 15) * 16;
    }
    const float* sw = A.wscale + t.e * A.wscale_stride;

    // NB of the tile's 32-row token tiles hold rows
    auto run = [&](auto nb) {
        constexpr int NB = decltype(nb)::value;
        // stages in flight: two where the registers allow it and a workgroup is
        // alone on its CU (500 tokens, 6144 -> 2048: 15.2 us against 17.2)
        constexpr int D = BM <= 64 ? 2 : 1;
        u32x4 x[D][NB][XW], w[D][2][4];
        auto load_tokens = [&](int d, int s) {
            int k = min(s, ns - 1) * kStageK + (lane & 7) * 16;
            if (k >= Kp) k = 0;                  // the weights there are zero
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int h = 0; h < XW; ++h)
                    x[d][i][h] = *reinterpret_cast<const u32x4*>(xp[i][h] + k);
        };
        auto put_tokens = [&](int d, int buf) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int h = 0; h < XW; ++h)
                    *reinterpret_cast<u32x4*>(tok[buf] + (i * 32 + h * 8) * kStageK + xat) =
                        x[d][i][h];
        };
        // The weights of input step j are reloaded, D stages ahead, as soon as
        // they are multiplied: registers for no more than what is in flight.
        auto load_w = [&](int d, int s, int j) {
            s = min(s, ns - 1);                  // past the end: the last again
#pragma unroll
            for (int c = 0; c < 2; ++c)
                w[d][c][j] = *reinterpret_cast<const u32x4*>(wp[c] + (int64_t)s * 2048 + j * 512);
        };
        i32x16 acc[NB][2];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][c][v] = 0;
#pragma unroll
        for (int d = 0; d < D; ++d) {
            load_tokens(d, sa + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                keep_order();                    // the waits below go by it
                load_w(d, sa + d, j);
            }
            keep_order();
        }
        put_tokens(0, 0);
        // stage i0 of the part, whose weights lie in set d
        auto stage = [&](int i0, auto dc) {
            constexpr int d = decltype(dc)::value;
            lds_barrier();
            if (KP > 1 && sa + i0 >= se) return;       // a shorter part: only the barrier
            load_tokens(d, sa + i0 + D);
            const uint8_t* base = tok[i0 & 1] + col * kStageK;
            u32x4 a[2][NB];
            auto read_a = [&](int j) {
                const int at = ((2 * j + (lane >> 5)) ^ (lane & 7)) * 16;
#pragma unroll
                for (int i = 0; i < NB; ++i)
                    a[j & 1][i] = *reinterpret_cast<const u32x4*>(base + i * 32 * kStageK + at);
            };
            read_a(0);
            keep_order();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j < 3) read_a(j + 1);
                else put_tokens((d + 1) % D, (i0 + 1) & 1);
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        acc[i][c] = mfma_i8_32(a[j & 1][i], w[d][c][j], acc[i][c]);
                load_w(d, sa + i0 + D, j);
                // one LDS access of the next step between every two products
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    if (j < 3) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                    else __builtin_amdgcn_sched_group_barrier(0x200, XW, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
                }
                __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
                keep_order();
            }
        };
        int i0 = 0;
        if constexpr (D == 2) {
            for (; i0 + 1 < steps; i0 += 2) {
                stage(i0, std::integral_constant<int, 0>{});
                stage(i0 + 1, std::integral_constant<int, 1>{});
            }
        }
        for (; i0 < steps; ++i0) stage(i0, std::integral_constant<int, 0>{});
        if constexpr (KP > 1) {
            // int32 sums: the same bits in any order
            int32_t* own = sums + wave * (BM * 64) + lane;
            if (part == 0) {
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            own[((i * 2 + c) * 16 + v) * 64] = acc[i][c][v];
            }
            __syncthreads();
            if (part > 0) {
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            __hip_atomic_fetch_add(&own[((i * 2 + c) * 16 + v) * 64], acc[i][c][v],
                                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            }
            __syncthreads();
        }

        // lane: rows 32 i + 8 (v >> 2) + 4 (lane >> 5) + (v & 3) of its column
        auto rows = [&](auto&& f) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const int row = 32 * i + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
                    if (KP > 1 && v / (16 / KP) != part) continue;   // the parts share the rows
                    if (row >= left) continue;
                    if constexpr (KP > 1) {
                        const int32_t* own = sums + wave * (BM * 64) + lane;
                        f(split(qs[row]), own[(i * 32 + v) * 64], own[(i * 32 + 16 + v) * 64],
                          (first + row) * A.ld_out);
                    } else {
                        f(split(qs[row]), acc[i][0][v], acc[i][1][v], (first + row) * A.ld_out);
                    }
                }
        };
        if constexpr (PAIR) {
            const int ch = g0 * 8 + col;
            if (ch >= A.N) return;
            const Scale sg = split(sw[ch]), su = split(sw[A.N + ch]);
            float* h = static_cast<float*>(A.out) + ch;
            rows([&](Scale q, int g, int u, int64_t at) {
                h[at] = silu_mul(scaled(q, sg, g), scaled(q, su, u));
            });
        } else {
            const int ch = g0 * 16 + 2 * col;
            if (ch >= A.N) return;
            const bool two = ch + 1 < A.N;
            const Scale s0 = split(sw[ch]), s1 = split(two ? sw[ch + 1] : 0.f);
            const float b0 = A.bias ? A.bias[ch] : 0.f, b1 = A.bias && two ? A.bias[ch + 1] : 0.f;
            auto store = [&](auto zero) {
                using T = decltype(zero);
                typedef T T2 __attribute__((ext_vector_type(2)));
                T* o = static_cast<T*>(A.out) + ch;
                rows([&](Scale q, int a0, int a1, int64_t at) {
                    const T y0 = as_type<T>(scaled(q, s0, a0) + b0);
                    const T y1 = as_type<T>(scaled(q, s1, a1) + b1);
                    if (pairs) {
                        *reinterpret_cast<T2*>(o + at) = T2{y0, y1};
                    } else {
                        o[at] = y0;
                        if (two) o[at + 1] = y1;
                    }
                });
            };
            if (A.out_dtype == MOE_DT_F32) store(0.f);
            else if (A.out_dtype == MOE_DT_BF16) store((__bf16)0.f);
            else store((_Float16)0.f);
        }
    };
    const int nb = (left + 31) / 32;
    if constexpr (NT == 1) {
        run(std::integral_constant<int, 1>{});
    } else if constexpr (NT == 2) {
        if (nb == 1) run(std::integral_constant<int, 1>{});
        else run(std::integral_constant<int, 2>{});
    } else {
        if (nb == 1) run(std::integral_constant<int, 1>{});
        else if (nb == 2) run(std::integral_constant<int, 2>{});
        else if (nb == 3) run(std::integral_constant<int, 3>{});
        else run(std::integral_constant<int, 4>{});
    }
}

template <int BM, int CW, int KP>
void launch(const I8Pass& p, bool pair, int ngroups, int64_t nm, hipStream_t s) {
    const int nnt = (ngroups + 4 * CW - 1) / (4 * CW);
    const unsigned grid = (unsigned)round_up(nm * nnt, 8 * kRun);
    // two neighbouring channels in one store
    const uintptr_t two = p.out_dtype == MOE_DT_F32 ? 8 : 4;
    const bool pairs = p.N % 2 == 0 && p.ld_out % 2 == 0 &&
                       reinterpret_cast<uintptr_t>(p.out) % two == 0;
    if (pair) k_gemm_i8<true, BM, CW, KP><<<grid, 64 * CW * KP, 0, s>>>(p, ngroups, nnt, pairs);
    else k_gemm_i8<false, BM, CW, KP><<<grid, 64 * CW * KP, 0, s>>>(p, ngroups, nnt, pairs);
}

}  // namespace

int launch_gemm_i8(const I8Pass& p, bool pair, void* stream) {
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int ngroups = (int)(round_up(p.N, 16) / 16) * (pair ? 2 : 1);
    const int64_t rows = p.T * p.k, used = p.offsets ? (p.E < rows ? p.E : rows) : 1;
    const int64_t mean = rows / used + (rows % used != 0);      // rows of a matrix
    // The largest tile that still makes about a workgroup for every CU.  Routed
    // experts' weights are streamed, once for each of an expert's tiles: a tile
    // that holds most experts whole (4 times the mean rows is not too large:
    // 2048 tokens on 256 experts, 64 rows each, 1.80 ms in tiles of 128 rows
    // against 1.99 in 64); one matrix's tiles are no larger than twice its rows.
    auto tiles = [&](int bm) { return p.offsets ? rows / bm + used : (rows + bm - 1) / bm; };
    auto fits = [&](int bm, int cw) {
        return (bm == 32 || mean > (p.offsets ? bm / 4 : bm / 2)) &&
               used * ((mean + bm - 1) / bm) * ((ngroups + 4 * cw - 1) / (4 * cw)) >= 160;
    };
    if (fits(128, 4)) launch<128, 4, 1>(p, pair, ngroups, tiles(128), s);
    else if (fits(64, 4)) launch<64, 4, 1>(p, pair, ngroups, tiles(64), s);
    else if (fits(64, 2)) launch<64, 2, 2>(p, pair, ngroups, tiles(64), s);
    else if (fits(32, 4)) launch<32, 4, 1>(p, pair, ngroups, tiles(32), s);
    else if (fits(32, 2)) launch<32, 2, 2>(p, pair, ngroups, tiles(32), s);
    else launch<32, 1, 4>(p, pair, ngroups, tiles(32), s);
    MOEQ_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace moeq
