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

template <int DT, bool TOP>
__global__ __launch_bounds__(kThreads) void k_slice(LogArgs A) {
    constexpr int B = DT == MOE_DT_F32 ? 4 : 2;
    __shared__ uint32_t order[kThreads];
    __shared__ float wred[3][kWaves];
    __shared__ uint32_t bound[2];                            // order and place of the bound
    __shared__ int ncol, ncand;
    __shared__ int col_of[kCols];
    __shared__ __attribute__((aligned(16))) uint8_t cols[TOP ? kCols * kChunks * 8 * B : 16];
    __shared__ uint64_t cand[TOP ? kCols * kChunks * 8 : 1];
    const moe_logprobs& P = A.P;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t = A.t0 + blockIdx.x / A.S;
    const int slice = blockIdx.x % A.S;
    const int v0 = slice * kSlice;
    const char* row = static_cast<const char*>(P.logits) + t * P.ld * B;

    // ------------------------------------------------ the slice, and its largest
    Raw8 x[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int v = v0 + (c * kThreads + tid) * 8;
        if (v + 8 <= P.V) {
            x[c] = load_raw8<true, true>(row, DT, v);
        } else {
            // past the row: -inf
            const uint32_t none = DT == MOE_DT_F32 ? 0xff800000u
                                  : DT == MOE_DT_BF16 ? 0xff80ff80u : 0xfc00fc00u;
            x[c].a = x[c].b = u32x4{none, none, none, none};
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
    float best = -__builtin_inff();
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) best = fmaxf(best, elem_of<DT>(x[c], e));
    if constexpr (TOP) order[tid] = order_of(best);
    float m = best;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    if (lane == 0) wred[0][wave] = m;
    if (tid == 0) ncol = ncand = 0;
    __syncthreads();
    m = wred[0][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, wred[0][w]);
    const float mx = m;
    if (m == -__builtin_inff()) m = 0.f;         // nothing but masked ones: every term is 0

    // ------------------------------------------------ a bound that the n best reach
    if constexpr (TOP) {
        if (wave == 0) {
            uint32_t o[kWaves];
#pragma unroll
            for (int i = 0; i < kWaves; ++i) o[i] = order[i * 64 + lane];
            auto reach = [&](uint32_t b) {
                int n = 0;
#pragma unroll
                for (int i = 0; i < kWaves; ++i) n += __popcll(__ballot(o[i] >= b));
                return n;
            };
            // lo is reached by more than kCols maxima or by all there are, hi by fewer than n
            uint32_t lo = 1u, place = 0xffffffffu;
            int n = reach(lo);
            if (n > kCols) {
                uint32_t hi = mono_bits(mx) + 1u;
                while (hi - lo > 1u) {
                    const uint32_t mid = lo + (hi - lo) / 2;
                    n = reach(mid);
                    if (n < P.top) {
                        hi = mid;
                    } else {
                        lo = mid;
                        if (n <= kCols) break;
                    }
                }
                if (n < P.top || n > kCols) n = reach(lo);
                if (n > kCols) {
                    // More threads than kCols whose largest is exactly lo: those with the
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
                                        order_of(load_elem(row, DT, v0 + at)) == lo)
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
                    place = ph;          // places are distinct: exactly `more` lie below it
                }
            }
            if (lane == 0) {
                bound[0] = lo;
                bound[1] = place;
            }
        }
    }

    // ------------------------------------------------ the sums
    const float k = scale_of(P, t) * 1.44269504088896340736f;
    float s = 0.f, d = 0.f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float z = (elem_of<DT>(x[c], e) - m) * k;
            const float p = __builtin_amdgcn_exp2f(z);
            s += p;
            d = __builtin_fmaf(p, fmaxf(z, -0x1p100f), d);     // a masked one: 0 * -inf
        }
    s = wave_sum(s);
    d = wave_sum(d);
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
        A.stat[at] = SliceStat{mx, ss, dd, 0.f};
    }
    if constexpr (!TOP) return;

    // ------------------------------------------------ the n best
    const uint32_t lo = bound[0], place = bound[1];
    auto reaches = [&](float v, uint32_t p) {
        const uint32_t o = order_of(v);
        return o > lo || (o == lo && p < place);
    };
    if (order_of(best) >= lo) {
        bool any = place == 0xffffffffu || order_of(best) > lo;
        if (!any) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    any = any || reaches(elem_of<DT>(x[c], e),
                                         (uint32_t)((c * kThreads + tid) * 8 + e));
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
    for (int i = tid; i < nc; i += kThreads) {
        const int place0 = ((i % kChunks) * kThreads + col_of[i / kChunks]) * 8;
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

// One wave per row: lane s holds slice s.
__global__ __launch_bounds__(64) void k_join(LogArgs A) {
    __shared__ uint64_t list[kLogprobSlices * MOE_MAX_TOP];
    const moe_logprobs& P = A.P;
    const int lane = threadIdx.x;
    const int64_t t = A.t0 + blockIdx.x;
    const bool in = lane < A.S;
    const int64_t at = t * A.S + (in ? lane : 0);
    const float NaN = __uint_as_float(0x7fc00000u), inf = __builtin_inff();
    const SliceStat st = A.stat[at];
    for (int i = lane; i < A.S * P.top; i += 64) list[i] = A.keys[t * A.S * P.top + i];
    const float sc = scale_of(P, t), k = sc * 1.44269504088896340736f;
    float M = in ? st.max : -inf;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor(M, off));
    const bool empty = M == -inf;
    float s = 0.f, d = 0.f;
    if (in) {
        // a slice of masked logits has S = 0; NaN of any slice stays
        const float z = st.max > -inf ? (st.max - M) * k : 0.f, f = __builtin_amdgcn_exp2f(z);
        s = st.sum * f;
        d = f * (st.dot + fmaxf(z, -0x1p100f) * st.sum);
    }
    s = wave_sum(s);
    d = wave_sum(d);
    const bool bad = !(s >= 0.f);
    const float logS = logf(s);
    auto logprob = [&](float x) {
        if (bad) return NaN;
        return empty || x == -inf ? -inf : (x - M) * sc - logS;
    };
    if (lane == 0 && P.entropy)
        P.entropy[t] = bad ? NaN : empty ? 0.f : fmaxf(logS - 0.69314718055994530942f * (d / s), 0.f);
    if (P.ids) {
        for (int j = lane; j < P.m; j += 64) {
            const int64_t id = P.id_bits == 64 ? static_cast<const int64_t*>(P.ids)[t * P.m + j]
                                               : static_cast<const int32_t*>(P.ids)[t * P.m + j];
            P.logprob[t * P.m + j] =
                id >= 0 && id < P.V ? logprob(load_elem(P.logits, P.dtype, t * P.ld + id)) : NaN;
        }
    }
    __syncthreads();
    uint64_t head = P.top && in ? list[lane * P.top] : 0ull;
    int taken = 0;
    int my_id = -1;
    float my_lp = bad ? NaN : -inf;
    for (int j = 0; j < P.top; ++j) {
        const uint32_t hi = (uint32_t)(head >> 32), lo = (uint32_t)head;
        const uint32_t best_hi = wave_max_u32(hi);
        if (best_hi == 0u) break;
        const uint32_t best_lo = wave_max_u32(hi == best_hi ? lo : 0u);
        if (lane == j) {
            my_id = (int)(0xffffffffu - best_lo);
            my_lp = logprob(mono_float(best_hi));
        }
        if (hi == best_hi && lo == best_lo) {
            head = ++taken < P.top ? list[lane * P.top + taken] : 0ull;
        }
    }
    if (lane < P.top) {
        P.top_ids[t * P.top + lane] = bad ? -1 : my_id;
        P.top_logprob[t * P.top + lane] = my_lp;
    }
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
        auto go = [&](auto top) {
            constexpr bool TOP = decltype(top)::value;
            if (P.dtype == MOE_DT_F32) k_slice<MOE_DT_F32, TOP><<<n * S, kThreads, 0, s>>>(A);
            else if (P.dtype == MOE_DT_BF16) k_slice<MOE_DT_BF16, TOP><<<n * S, kThreads, 0, s>>>(A);
            else k_slice<MOE_DT_F16, TOP><<<n * S, kThreads, 0, s>>>(A);
        };
        if (P.top) go(std::true_type{});
        else go(std::false_type{});
        k_join<<<n, 64, 0, s>>>(A);
    }
    MOEQ_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace moeq
