// Log probabilities of given tokens, the entropy and the best tokens of rows of
// logits.  Per row, z = scale * x, over the tokens of its V logits x:
//
//   M = max x,  S = sum e^(scale (x - M)),  E = sum e^(scale (x - M)) scale (x - M)
//   log p(v) = scale (x_v - M) - log S,  entropy = log S - E / S
//   the n largest x, equal ones by the lower id, with their log p
//
// Two launches.  The first cuts each row into slices of 16384 logits, one workgroup
// of 512 threads each, which loads its slice into registers (32 logits a thread, all
// loads in flight at once), reduces it to (M, S, E) and picks its n best; the
// second joins a row's slices in one wave.  The cut follows V alone, so that a
// row's bits do not depend on how many rows there are.
//
// The n best of a slice: the n threads with the largest maxima hold them all, so a
// bisection over the threads' maxima (ballots of one wave) finds a bound that at
// least n and at most kCols maxima reach; those threads' logits go through LDS, where
// the few that reach the bound are collected and ranked by counting.
//
// HBM bounds large batches: 2048 rows of 131072 in bf16 take 84 us without best tokens
// (6.4 TB/s), 109 with 8 of them, since a workgroup searches when its loads are done.  A
// row alone is two launches (5.8 and 3.3 us of kernels), 32 rows of fp32 a single wave of
// workgroups (8.6 and 5.0).
#include "elem_dev.h"
#include "topk_dev.h"

namespace moeq {

namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64, kChunks = 4;
constexpr int kSlice = kLogprobSlice;
constexpr int kCols = 64;                       // threads whose logits are looked through
static_assert(kSlice == kThreads * kChunks * 8 && kCols >= MOE_MAX_TOP, "slices");

struct SliceStat {
    float max, sum, dot;   // M, S, E in log2 units; S NaN: a NaN or an infinity among them
    float pad;
};

struct LogArgs {
    moe_logprobs P;
    int64_t t0;
    int S;                 // slices of a row
    SliceStat* stat;       // [T][S]
    uint64_t* keys;        // [T][S][top], 0: none
};

__device__ __forceinline__ float scale_of(const moe_logprobs& P, int64_t t) {
    const float s = P.scale ? P.scale[t] : 1.f;
    return s > 0.f && s < __builtin_inff() ? s : __uint_as_float(0x7fc00000u);
}

// The scale in units of log2 e.  Past 2^128 / log2 e that leaves fp32's range where the scale
// does not: k is half of it, and an exponent k times its difference twice that.
struct ScaleLog2 {
    float k, twice;
    __device__ __forceinline__ explicit ScaleLog2(float s)
        : k(s * 1.44269504088896340736f), twice(1.f) {
        if (k < __builtin_inff()) return;
        k = 0.5f * s * 1.44269504088896340736f;
        twice = 2.f;
    }
};

// (x - M) k of x <= M, both finite, also where the difference leaves fp32's range.
__device__ __forceinline__ float diff_times(float x, float M, float k) {
    const float d = x - M;
    return d > -__builtin_inff() ? d * k : (0.5f * x - 0.5f * M) * k * 2.f;
}

// A logit's order: 0 for the masked ones (-inf; NaN too), which no list holds.
__device__ __forceinline__ uint32_t order_of(float x) {
    return x > -__builtin_inff() ? mono_bits(x) : 0u;
}

template <int DT>
__device__ __forceinline__ float elem_of(const Raw8& r, int e) {
    if constexpr (DT == MOE_DT_F32) {
        return __uint_as_float(e < 4 ? r.a[e & 3] : r.b[e & 3]);
    } else if constexpr (DT == MOE_DT_BF16) {
        const uint32_t w = r.a[e >> 1];
        return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
    } else {
        return (float)__builtin_bit_cast(f16x8, r.a)[e];
    }
}

// The largest and smallest of three; a NaN is not looked at.  (The compiler's own form
// of fmaxf first quiets every loaded value, an instruction more each.)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float r;
    asm("v_min3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// Over the wave, the same in every lane: DPP steps inside rows of 16 lanes, then the
// four rows.
template <class F>
__device__ __forceinline__ float wave_all(float v, F f) {
    auto step = [&](auto ctrl) {
        const int u = (int)__float_as_uint(v);
        v = f(v, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
                     u, u, decltype(ctrl)::value, 0xf, 0xf, false)));
    };
    step(std::integral_constant<int, 0xB1>{});
    step(std::integral_constant<int, 0x4E>{});
    step(std::integral_constant<int, 0x141>{});
    step(std::integral_constant<int, 0x140>{});
    auto lane = [&](int i) {
        return __uint_as_float(
            (uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), i));
    };
    return f(f(lane(0), lane(16)), f(lane(32), lane(48)));
}
__device__ __forceinline__ float all_max(float v) {
    return wave_all(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float all_sum(float v) {
    return wave_all(v, [](float a, float b) { return a + b; });
}

// 16-bit logits: 64 registers, so that four workgroups share a CU and some of them load
// while the others reduce (2048 rows of 131072 bf16, 8 best tokens: 109 us against 121).
// STREAM: logits that no cache holds.
template <int DT, bool TOP, bool STREAM>
__global__ __launch_bounds__(kThreads, DT == MOE_DT_F32 ? 4 : 8) void k_slice(LogArgs A) {
    constexpr int B = DT == MOE_DT_F32 ? 4 : 2;
    // the low bits of a logit's order that are the same in all of them
    constexpr int SH = DT == MOE_DT_F32 ? 0 : DT == MOE_DT_BF16 ? 16 : 13;
    __shared__ uint32_t order[TOP ? kThreads : 1];
    __shared__ float wred[3][kWaves];
    __shared__ uint32_t bound[2];                            // order and place of the bound
    __shared__ int ncol, ncand;
    __shared__ int col_of[kCols];
    __shared__ __attribute__((aligned(16))) uint8_t cols[TOP ? kCols * kChunks * 8 * B : 16];
    __shared__ uint64_t cand[TOP ? kCols * kChunks * 8 : 1];
    const moe_logprobs& P = A.P;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t t = A.t0 + blockIdx.x / A.S;
    const int slice = blockIdx.x % A.S;
    const int v0 = slice * kSlice;
    const char* row = static_cast<const char*>(P.logits) + t * P.ld * B;

    // asked for with the logits, not behind them (2048 rows: 118 -> 109 us)
    const ScaleLog2 scale(scale_of(P, t));
    const float k = scale.k, twice = scale.twice;

    // ------------------------------------------------ the slice, and its largest
    Raw8 x[kChunks];
    if (v0 + kSlice <= P.V) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
            x[c] = load_raw8<STREAM, true>(row, DT, v0 + (c * kThreads + tid) * 8);
    } else {
        // past the row: -inf
        const uint32_t none = DT == MOE_DT_F32 ? 0xff800000u
                              : DT == MOE_DT_BF16 ? 0xff80ff80u : 0xfc00fc00u;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int v = v0 + (c * kThreads + tid) * 8;
            x[c].a = x[c].b = u32x4{none, none, none, none};
            if (v + 8 <= P.V) {
                x[c] = load_raw8<STREAM, true>(row, DT, v);
            } else if (v < P.V) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (v + e >= P.V) continue;
                    if constexpr (DT == MOE_DT_F32) {
                        const uint32_t w = reinterpret_cast<const uint32_t*>(row)[v + e];
                        if (e < 4) x[c].a[e & 3] = w;
                        else x[c].b[e & 3] = w;
                    } else {
                        const uint32_t w = reinterpret_cast<const uint16_t*>(row)[v + e];
                        const uint32_t o = x[c].a[e >> 1];
                        x[c].a[e >> 1] = e & 1 ? (o & 0xffffu) | w << 16 : (o & 0xffff0000u) | w;
                    }
                }
            }
        }
    }
    // chunks that lie past the row add nothing (333 rows of 50257 fp16: 15.5 -> 14.2 us)
    auto past = [&](int c) { return c && v0 + c * kThreads * 8 >= P.V; };
    float best = -__builtin_inff(), least = __builtin_inff();
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        if (past(c)) continue;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float u = elem_of<DT>(x[c], e), v = elem_of<DT>(x[c], e + 1);
            best = max3(best, u, v);
            least = min3(least, u, v);
        }
    }
    if constexpr (DT != MOE_DT_F32) {
        // converted again below: 16 registers of 16-bit logits live on, not 32
#pragma unroll
        for (int c = 0; c < kChunks; ++c) asm volatile("" : "+v"(x[c].a));
    }
    if constexpr (TOP) order[tid] = order_of(best);
    const float wmax = all_max(best);
    if (lane == 0) wred[0][wave] = wmax;
    if (tid == 0) ncol = ncand = 0;
    __syncthreads();
    float m = wred[0][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, wred[0][w]);
    const float mx = m;
    if (m == -__builtin_inff()) m = 0.f;         // nothing but masked ones: every term is 0

    // ------------------------------------------------ a bound that the n best reach
    if constexpr (TOP) {
        if (wave == 0) {
            // The largest of 64 groups of threads: the n-th of these is reached by n
            // logits at least, and by few threads more than n.  A bisection between the
            // smallest and the largest group; it ends where a quarter too many reach it.
            uint32_t o[kWaves], top = 0u;
#pragma unroll
            for (int i = 0; i < kWaves; ++i) {
                o[i] = order[i * 64 + lane] >> SH;
                top = max(top, o[i]);
            }
            auto reach = [&](uint32_t b) {
                int n = 0;
#pragma unroll
                for (int i = 0; i < kWaves; ++i) n += __popcll(__ballot(o[i] >= b));
                return n;
            };
            // lo is reached by n groups at least (or by all there are), hi by fewer
            uint32_t lo = max(~wave_max_u32(~top), 1u), place = 0xffffffffu;
            const uint32_t end = (order_of(mx) >> SH) + 1u;
            uint32_t hi = end;
            int n = __popcll(__ballot(top >= lo));
            while (n > P.top + P.top / 4 && hi - lo > 1u) {
                const uint32_t mid = lo + (hi - lo) / 2;
                const int k = __popcll(__ballot(top >= mid));
                if (k < P.top) {
                    hi = mid;
                } else {
                    lo = mid;
                    n = k;
                }
            }
            n = reach(lo);
            if (n > kCols) {
                // Too many threads: the same over all of them.
                hi = end;
                while (hi - lo > 1u) {
                    const uint32_t mid = lo + (hi - lo) / 2;
                    const int k = reach(mid);
                    if (k < P.top) {
                        hi = mid;
                    } else {
                        lo = mid;
                        n = k;
                        if (k <= kCols) break;
                    }
                }
            }
            if (n > kCols) {
                // More than kCols threads whose largest is exactly lo: those with the
                // lowest places hold the best of them.  place: the bound of the places.
                const int more = P.top - reach(lo + 1u);
                uint32_t pl = 0u, ph = (uint32_t)kSlice;        // fewer than more below pl
                uint32_t first[kWaves];
#pragma unroll
                for (int i = 0; i < kWaves; ++i) {
                    // the lowest place of a thread's logits that equal lo
                    first[i] = 0xffffffffu;
                    if (o[i] == lo) {
                        for (int c = kChunks - 1; c >= 0; --c)
                            for (int e = 7; e >= 0; --e) {
                                const int at = (c * kThreads + i * 64 + lane) * 8 + e;
                                if (v0 + at < P.V &&
                                    order_of(load_elem(row, DT, v0 + at)) >> SH == lo)
                                    first[i] = (uint32_t)at;
                            }
                    }
                }
                while (ph - pl > 1u) {
                    const uint32_t mid = pl + (ph - pl) / 2;
                    int k = 0;
#pragma unroll
                    for (int i = 0; i < kWaves; ++i) k += __popcll(__ballot(first[i] < mid));
                    if (k < more) pl = mid;
                    else ph = mid;
                }
                place = ph;              // places are distinct: exactly `more` lie below it
            }
            if (lane == 0) {
                bound[0] = lo;
                bound[1] = place;
            }
        }
    }

    // ------------------------------------------------ the sums
    // z = x k - m k in one instruction.  What m k loses in its rounding (under 2^-4) is the
    // same for every term of the slice and put back at the end; past 2^20 it could be more
    // than an exponent holds, and z is (x - m) k, as it is for the largest scales.  Terms
    // whose z is -inf, as a masked one's is or may overflow to, have p = 0 and add nothing to
    // d: a wave that may hold one bounds z.
    const float mk = m * k, rest = __builtin_fmaf(m, k, -mk);
    const bool far = !(fabsf(mk) < 0x1p20f) || twice != 1.f;
    const bool low = __any(!(least * k > -0x1p100f));
    float s = 0.f, d = 0.f;
    auto sums = [&](auto apart, auto bounded) {
        constexpr bool APART = decltype(apart)::value, BOUNDED = decltype(bounded)::value;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            if (past(c)) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = elem_of<DT>(x[c], e);
                float z = APART ? (v - m) * k * twice : __builtin_fmaf(v, k, -mk);
                const float p = __builtin_amdgcn_exp2f(z);
                s += p;
                if constexpr (BOUNDED) z = fmaxf(z, -0x1p100f);    // 0 * -inf
                d = __builtin_fmaf(p, z, d);
            }
        }
    };
    const std::true_type yes;
    const std::false_type no;
    if (far) sums(yes, yes);
    else if (low) sums(no, yes);
    else sums(no, no);
    s = all_sum(s);
    d = all_sum(d);
    if (lane == 0) {
        wred[1][wave] = s;
        wred[2][wave] = d;
    }
    __syncthreads();
    const int64_t at = t * A.S + slice;
    if (tid == 0) {
        float ss = 0.f, dd = 0.f;
        for (int w = 0; w < kWaves; ++w) {
            ss += wred[1][w];
            dd += wred[2][w];
        }
        if (!far) {
            dd = __builtin_fmaf(-rest, ss, dd);
            const float g = __builtin_amdgcn_exp2f(-rest);
            ss *= g;
            dd *= g;
        }
        A.stat[at] = SliceStat{mx, ss, dd, 0.f};
    }
    if constexpr (!TOP) return;

    // ------------------------------------------------ the n best
    const uint32_t lo = bound[0], place = bound[1];
    auto reaches = [&](float v, uint32_t p) {
        const uint32_t o = order_of(v) >> SH;
        return o > lo || (o == lo && p < place);
    };
    const uint32_t mine = order_of(best) >> SH;
    if (mine >= lo) {
        bool any = place == 0xffffffffu || mine > lo;
        if (!any) {
            for (int c = 0; c < kChunks; ++c)
                for (int e = 0; e < 8; ++e) {
                    const int p = (c * kThreads + tid) * 8 + e;
                    any = any || (v0 + p < P.V && reaches(load_elem(row, DT, v0 + p), (uint32_t)p));
                }
        }
        if (any) {
            const int j = atomicAdd(&ncol, 1);               // the order changes no result
            if (j < kCols) {
                col_of[j] = tid;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    uint8_t* q = cols + (j * kChunks + c) * 8 * B;
                    *reinterpret_cast<u32x4*>(q) = x[c].a;
                    if constexpr (DT == MOE_DT_F32) *reinterpret_cast<u32x4*>(q + 16) = x[c].b;
                }
            }
        }
    }
    __syncthreads();
    const int nc = min(ncol, kCols) * kChunks;
    if (tid < nc) {
        const int i = tid, place0 = ((i % kChunks) * kThreads + col_of[i / kChunks]) * 8;
        Raw8 r;
        r.a = *reinterpret_cast<const u32x4*>(cols + i * 8 * B);
        if constexpr (DT == MOE_DT_F32) r.b = *reinterpret_cast<const u32x4*>(cols + i * 8 * B + 16);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = elem_of<DT>(r, e);
            if (reaches(v, (uint32_t)(place0 + e)))
                cand[atomicAdd(&ncand, 1)] = make_key(v, v0 + place0 + e);
        }
    }
    __syncthreads();
    const int n = ncand;
    uint64_t* out = A.keys + at * P.top;
    for (int i = tid; i < n; i += kThreads) {
        const uint64_t mine = cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += cand[j] > mine;
        if (rank < P.top) out[rank] = mine;
    }
    for (int i = n + tid; i < P.top; i += kThreads) out[i] = 0ull;
}
static_assert(kCols * kChunks <= kThreads, "a chunk a thread");

constexpr int kFlat = 512;                      // threads of a flat join, two a key

// One workgroup per row: a wave, in which lane s holds slice s, or, for the best tokens of
// few slices, eight (FLAT).
template <bool FLAT>
__global__ __launch_bounds__(FLAT ? kFlat : 64) void k_join(LogArgs A) {
    __shared__ uint64_t list[FLAT ? kFlat / 2 : kLogprobSlices * MOE_MAX_TOP];
    const moe_logprobs& P = A.P;
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t t = A.t0 + blockIdx.x;
    const bool in = lane < A.S;
    const float NaN = __uint_as_float(0x7fc00000u), inf = __builtin_inff();
    const SliceStat st = A.stat[t * A.S + (in ? lane : 0)];
    for (int i = tid; i < A.S * P.top; i += FLAT ? kFlat : 64)
        list[i] = A.keys[t * A.S * P.top + i];
    auto id_of = [&](int j) {
        return P.id_bits == 64 ? static_cast<const int64_t*>(P.ids)[t * P.m + j]
                               : (int64_t) static_cast<const int32_t*>(P.ids)[t * P.m + j];
    };
    auto logit_of = [&](int64_t id) {
        return id >= 0 && id < P.V ? load_elem(P.logits, P.dtype, t * P.ld + id) : NaN;
    };
    // the given tokens' logits are on their way before the slices are joined
    const float given = lane < P.m ? logit_of(id_of(lane)) : 0.f;
    const float sc = scale_of(P, t);
    const ScaleLog2 scale(sc);
    const float M = all_max(in ? st.max : -inf);
    const bool empty = M == -inf;
    float s = 0.f, d = 0.f;
    if (in) {
        // a slice of masked logits has S = 0; NaN of any slice stays
        const float z = st.max > -inf ? diff_times(st.max, M, scale.k) * scale.twice : 0.f;
        const float f = __builtin_amdgcn_exp2f(z);
        s = st.sum * f;
        d = f * (st.dot + fmaxf(z, -0x1p100f) * st.sum);
    }
    s = all_sum(s);
    d = all_sum(d);
    const bool bad = !(s >= 0.f) || d != d;
    const float logS = logf(s);
    auto logprob = [&](float x) {
        if (bad || x != x) return NaN;
        return empty || x == -inf ? -inf : diff_times(x, M, sc) - logS;
    };
    if (tid == 0 && P.entropy)
        P.entropy[t] = bad ? NaN : empty ? 0.f : fmaxf(logS - 0.69314718055994530942f * (d / s), 0.f);
    if (tid < 64) {
        if (lane < P.m) P.logprob[t * P.m + lane] = logprob(given);
        for (int j = lane + 64; j < P.m; j += 64)
            P.logprob[t * P.m + j] = logprob(logit_of(id_of(j)));
    }
    if (P.top == 0) return;
    __syncthreads();
    auto put = [&](int place, uint64_t key) {
        const bool none = bad || key == 0ull;
        P.top_ids[t * P.top + place] = none ? -1 : (int)(0xffffffffu - (uint32_t)key);
        P.top_logprob[t * P.top + place] =
            bad ? NaN : none ? -inf : logprob(mono_float((uint32_t)(key >> 32)));
    };
    if constexpr (FLAT) {
        // A key's place among all of them: how many are larger, half of them counted by
        // either of its threads (32 rows, 20 best of 8 slices: 4.8 us against 5.5 with one).
        const int n = A.S * P.top, i = tid >> 1, half = tid & 1;
        const uint64_t key = i < n ? list[i] : 0ull;
        const int all = __syncthreads_count(half == 0 && key != 0ull);
        if ((tid & ~63) >= 2 * n) return;
        int place = 0;
#pragma unroll 8
        for (int j = half; j < n; j += 2) place += list[j] > key;
        place += __shfl_xor(place, 1);
        if (half == 0 && key != 0ull && place < P.top) put(place, key);
        if (tid >= all && tid < P.top) put(tid, 0ull);
        return;
    }
    // The slices' lists are in order: the largest head is the next best token, `top` times.
    uint64_t head = in ? list[lane * P.top] : 0ull, mine = 0ull;
    int taken = 0;
    for (int j = 0; j < P.top; ++j) {
        const uint64_t next = in && taken + 1 < P.top ? list[lane * P.top + taken + 1] : 0ull;
        const uint32_t hi = (uint32_t)(head >> 32), lo = (uint32_t)head;
        const uint32_t best_hi = wave_max_u32(hi);
        if (best_hi == 0u) break;
        const uint64_t tied = __ballot(hi == best_hi);
        uint32_t best_lo;
        if (__popcll(tied) == 1)
            best_lo = (uint32_t)__builtin_amdgcn_readlane(lo, __ffsll((unsigned long long)tied) - 1);
        else
            best_lo = wave_max_u32(hi == best_hi ? lo : 0u);
        if (lane == j) mine = (uint64_t)best_hi << 32 | best_lo;
        if (hi == best_hi && lo == best_lo) {
            head = next;
            ++taken;
        }
    }
    if (lane < P.top) put(lane, mine);
}

}  // namespace

int launch_logprobs(const moe_logprobs& P, int64_t T, void* ws, void* stream) {
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int S = (int)((P.V + kSlice - 1) / kSlice);
    LogArgs A{P, 0, S, static_cast<SliceStat*>(ws), nullptr};
    A.keys = reinterpret_cast<uint64_t*>(A.stat + T * S);
    const int64_t most = rows_of_launch(kWaves) / S;
    for (A.t0 = 0; A.t0 < T; A.t0 += most) {
        const unsigned n = (unsigned)(T - A.t0 < most ? T - A.t0 : most);
        auto go = [&](auto top, auto stream) {
            constexpr bool TOP = decltype(top)::value, STREAM = decltype(stream)::value;
            if (P.dtype == MOE_DT_F32)
                k_slice<MOE_DT_F32, TOP, STREAM><<<n * S, kThreads, 0, s>>>(A);
            else if (P.dtype == MOE_DT_BF16)
                k_slice<MOE_DT_BF16, TOP, STREAM><<<n * S, kThreads, 0, s>>>(A);
            else
                k_slice<MOE_DT_F16, TOP, STREAM><<<n * S, kThreads, 0, s>>>(A);
        };
        // More logits than the caches hold are read past them (2048 rows of 131072 bf16, no
        // best tokens: 84.5 us against 88.3, 8 of them: 110 against 115); fewer may be found
        // there (32 rows of fp32, 20 best tokens: 12.5 us against 13.3).
        const bool large = T * P.V * (P.dtype == MOE_DT_F32 ? 4 : 2) >= (int64_t)1 << 28;
        auto by = [&](auto top) {
            if (large) go(top, std::true_type{});
            else go(top, std::false_type{});
        };
        if (P.top) by(std::true_type{});
        else by(std::false_type{});
        // Few rows of up to 256 keys: two threads each (32 rows, 20 best of 8 slices: 4.8 us
        // against 6.6 with one best token after the other; 2048 rows: 8.9 against 5.2).
        if (P.top && S * P.top <= kFlat / 2 && T <= 512) k_join<true><<<n, kFlat, 0, s>>>(A);
        else k_join<false><<<n, 64, 0, s>>>(A);
    }
    MOEQ_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace moeq
