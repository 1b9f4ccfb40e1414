// The norms before and after a block, fused with the block's gate, the
// residual scales, a routed layer's gated sum and the 8-bit code of the
// result.  Per token row, in fp32:
//
//   b  = y[t]   or   sum_j w[t, j] * y[inv_perm[t*k + j]] (ascending j)
//                    + shared_gate[t] * y_shared[t]
//   p  = post_w ? b / sqrt(mean(b^2) + eps) * (w_offset + post_w) : b
//   r' = r_scale * r + y_scale * gate * p              -> r_out (rounded once)
//   n  = r' / sqrt(mean(r'^2) + eps) * (w_offset + pre_w)     -> n_out
//   codes of n and their scale                           -> q_out, q_scale
//
// A workgroup owns a row and keeps it in registers (NCH chunks of V elements
// per thread), so every operand is read once and every result written once; the
// reductions (b^2, r'^2, max |n|) go through LDS.  HBM bounds large batches: at
// 4096 tokens, H 6144, bf16, rows that no cache holds, the norm alone moves 101
// MB in 25 us, norm after + gate + residual + norm before 201 MB in 47 us, the
// gated sum of 8 rows + residual + norm 554 MB in 106 us (4.0, 4.3 and 5.2 TB/s;
// a plain copy reaches 4.8).  Small ones are bound by a launch and two or three
// dependent steps: 3.2 us for one token's norm, 6.7 for the gated sum of 8 tokens.
#include <type_traits>

#include "elem_dev.h"

namespace moeq {

namespace {

struct BlockRow {
    moe_block b;
    int64_t t0;     // the launch's first row
    int H, nw;      // nw: waves of a row
};

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ float uniform(float v) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

// COMB: slots of the gated sum that are in flight together, 0: y is a row.
// STREAM: more rows than the caches hold; results (1) and the rows of a gated
// sum (2) go past them.  Everything the row needs is loaded before the first reduction (EARLY), while
// it fits the registers of a workgroup of 1024 threads.
// ANY: rows that start off 16 bytes or end inside a chunk.  The last chunk then
// ends at the row's end and shares `lo` elements with the one before, which owns
// them: the other neither adds nor stores them (and may find them overwritten,
// where results go over operands).
template <int V, int NCH, int COMB, int STREAM, bool ANY>
__global__ __launch_bounds__(1024) void k_block(BlockRow A) {
    constexpr bool EARLY = V * NCH <= 8;
    constexpr int NE = EARLY ? NCH : 1;
    __shared__ float red[2][64];
    __shared__ uint32_t red_max[16];
    const moe_block& b = A.b;
    const int64_t t = A.t0 + blockIdx.x;
    const int H = A.H, nt = A.nw * 64;
    const bool has_y = COMB || b.y;
    float v[NCH][V];
    Raw<V> rr[NE], rp[NE], rg[NE], rn[NE];
    // a thread's elements at(c) + lo(c) .. at(c) + V: none past the row, where it
    // reads the last ones
    auto place = [&](int c) { return (c * nt + (int)threadIdx.x) * V; };
    auto at = [&](int c) { return min(place(c), H - V); };
    auto lo = [&](int c) { return place(c) - at(c); };
    auto load_r = [&](int c, Raw<V>& x) {
        if (b.r) x.template load<false, ANY>(b.r, b.r_dtype, t * b.ld_r + at(c));
    };
    auto load_p = [&](int c, Raw<V>& x) {
        if (b.post_w) x.template load<false, ANY>(b.post_w, b.w_dtype, at(c));
    };
    auto load_g = [&](int c, Raw<V>& x) {
        if (b.gate && b.gate_ld_h)
            x.template load<false, ANY>(b.gate, b.gate_dtype, t * b.gate_ld_t + at(c));
    };
    auto load_n = [&](int c, Raw<V>& x) {
        if (b.pre_w) x.template load<false, ANY>(b.pre_w, b.w_dtype, at(c));
    };
    const float gate1 = b.gate && !b.gate_ld_h ? load_elem(b.gate, b.gate_dtype, t * b.gate_ld_t)
                                               : 1.f;

    // ------------------------------------------------ the block's output
    Raw<V> ry[NCH];
    if constexpr (COMB == 0) {
        if (b.y) {
#pragma unroll
            for (int c = 0; c < NCH; ++c) ry[c].template load<false, ANY>(b.y, b.y_dtype, t * b.ld_y + at(c));
        }
    } else if (b.y_shared) {
#pragma unroll
        for (int c = 0; c < NCH; ++c)
            ry[c].template load<false, ANY>(b.y_shared, b.y_shared_dtype,
                                            t * b.ld_y_shared + at(c));
    }
    if constexpr (EARLY) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            load_r(c, rr[c]);
            load_p(c, rp[c]);
            load_g(c, rg[c]);
            load_n(c, rn[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int e = 0; e < V; ++e) v[c][e] = 0.f;
    if constexpr (COMB > 0) {
        for (int j0 = 0; j0 < b.k; j0 += COMB) {
            int64_t row[COMB];
            float wj[COMB];
#pragma unroll
            for (int u = 0; u < COMB; ++u) {
                const int64_t a = t * b.k + min(j0 + u, b.k - 1);
                row[u] = b.inv_perm[a] * b.ld_y;
                wj[u] = b.topk_w[a];
            }
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
                Raw<V> y[COMB];
#pragma unroll
                for (int u = 0; u < COMB; ++u)
                    y[u].template load<STREAM == 2, ANY>(b.y, b.y_dtype, row[u] + at(c));
#pragma unroll
                for (int u = 0; u < COMB; ++u) {
                    if (j0 + u >= b.k) break;
                    float f[V];
                    y[u].f32(b.y_dtype, f);
#pragma unroll
                    for (int e = 0; e < V; ++e) v[c][e] += wj[u] * f[e];
                }
            }
        }
        if (b.y_shared) {
            const float sg = b.shared_gate ? b.shared_gate[t] : 1.f;
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
                float f[V];
                ry[c].f32(b.y_shared_dtype, f);
#pragma unroll
                for (int e = 0; e < V; ++e) v[c][e] += sg * f[e];
            }
        }
    } else if (b.y) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) ry[c].f32(b.y_dtype, v[c]);
    }

    // ------------------------------------------------ the norm after
    // The sum of squares: by chunk, then 64 neighbouring chunks over lanes, then
    // these parts in order, or over lanes again where there are many: chains of at
    // most 30 sums, and one order whatever part of the row a wave holds.
    auto mean_square = [&](float* part, float k) {
        const int n64 = (H + 64 * V - 1) / (64 * V);
        float total = 0.f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            float ss = 0.f;
            if (lo(c) < V) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float x = ANY && e < lo(c) ? 0.f : v[c][e] * k;
                    ss += x * x;
                }
            }
            ss = wave_sum(ss);
            if (c == 0) total = ss;          // the whole row where it is one such part
            const int i = c * A.nw + ((int)threadIdx.x >> 6);
            if (n64 > 1 && i < n64 && (threadIdx.x & 63) == 0) part[i] = ss;
        }
        if (n64 > 1) {
            __syncthreads();
            total = 0.f;
            if (n64 <= 16) {
                for (int i = 0; i < n64; ++i) total += part[i];
            } else {
                for (int i = threadIdx.x & 63; i < n64; i += 64) total += part[i];
                total = wave_sum(total);
            }
        }
        return total / (float)H;
    };
    // 1 / sqrt(mean square + eps) of the row times `scale`, which is 1 unless the
    // squares leave fp32's range: past the top, where the largest magnitude is over
    // 2^56, 2^-80; below 2^-100, where squares that underflow might count and
    // magnitudes are under 2^-42, 2^100.  v * scale * rstd does not notice.  (The
    // test costs one token's norm 3.13 -> 3.20 us, norm after and before of 4096 x
    // 6144 bf16 47.3 -> 48.6.)
    float rstd = 1.f, scale = 1.f;
    auto norm = [&](float* part) {
        float ms = uniform(mean_square(part, 1.f) + b.eps);
        scale = 1.f;
        if (!(ms >= 0x1p-100f && ms < __builtin_inff())) {
            scale = ms < 1.f ? 0x1p100f : 0x1p-80f;
            __syncthreads();                 // part has been read
            ms = uniform(mean_square(part, scale) + b.eps * scale * scale);
        }
        rstd = 1.f / sqrtf(ms);
    };
    if (has_y && b.post_w) norm(red[0]);

    // ------------------------------------------------ gate, scales, residual
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        constexpr bool E = EARLY;
        Raw<V>& xr = rr[E ? c : 0];
        Raw<V>& xp = rp[E ? c : 0];
        Raw<V>& xg = rg[E ? c : 0];
        if constexpr (!E) {
            load_r(c, xr);
            load_p(c, xp);
            load_g(c, xg);
        }
        if (has_y) {
            float f[V];
            if (b.post_w) {
                xp.f32(b.w_dtype, f);
#pragma unroll
                for (int e = 0; e < V; ++e) v[c][e] = v[c][e] * scale * rstd * (b.w_offset + f[e]);
            }
            if (b.gate) {
                if (b.gate_ld_h) xg.f32(b.gate_dtype, f);
#pragma unroll
                for (int e = 0; e < V; ++e) v[c][e] *= b.gate_ld_h ? f[e] : gate1;
            }
#pragma unroll
            for (int e = 0; e < V; ++e) v[c][e] *= b.y_scale;
        }
        if (b.r) {
            float f[V];
            xr.f32(b.r_dtype, f);
#pragma unroll
            for (int e = 0; e < V; ++e)
                v[c][e] = has_y ? b.r_scale * f[e] + v[c][e] : b.r_scale * f[e];
        }
        if (b.r_out && lo(c) < V)
            store_from<V, (STREAM > 0), ANY>(b.r_out, b.r_dtype, t * b.ld_r_out + at(c), v[c],
                                             lo(c));
    }
    if (!b.n_out && !b.q_out) return;

    // ------------------------------------------------ the norm before the next
    if (b.pre_w) norm(red[1]);
    uint32_t amax = 0u;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        Raw<V>& xn = rn[EARLY ? c : 0];
        if constexpr (!EARLY) load_n(c, xn);
        if (b.pre_w) {
            float f[V];
            xn.f32(b.w_dtype, f);
#pragma unroll
            for (int e = 0; e < V; ++e) v[c][e] = v[c][e] * scale * rstd * (b.w_offset + f[e]);
        }
        if (lo(c) >= V) continue;
        if (b.n_out)
            store_from<V, (STREAM > 0), ANY>(b.n_out, b.n_dtype, t * b.ld_n + at(c), v[c], lo(c));
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (!ANY || e >= lo(c)) amax = max(amax, __float_as_uint(v[c][e]) & 0x7fffffffu);
    }
    if (!b.q_out) return;

    // ------------------------------------------------ its 8-bit code
    amax = block_max(amax, red_max, A.nw);
    const RowCode rc = row_code(amax);
    if (threadIdx.x == 0) b.q_scale[t] = rc.scale;
    int8_t* q = b.q_out + t * b.ld_q;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        if (lo(c) >= V) continue;
        if (V == 8 && (!ANY || lo(c) == 0)) {
            const uint2 u = {pack_codes4(&v[c][0], rc.mul), pack_codes4(&v[c][V / 2], rc.mul)};
            *reinterpret_cast<uint2*>(q + at(c)) = u;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (e >= lo(c)) q[at(c) + e] = code1(v[c][e], rc.mul);
        }
    }
    const int pad = (H + 63) / 64 * 64 - H;
    if ((int)threadIdx.x < pad) q[H + threadIdx.x] = 0;
}

template <int V, int NCH, bool ANY>
void launch(BlockRow& A, int64_t T, hipStream_t s) {
    constexpr int C = 4;
    // Results of 2M elements and more go past the caches (4096 rows of 6144 bf16
    // that were not in them: 26.2 -> 23.0 us for the norm alone, 116 -> 103 with
    // the gated sum of 8 rows each, which are then read past them too; fp32
    // rows are not: 194 us against 181).  A call that reads the results at once
    // finds less of them: residual + code + residual 98.8 us against 96.5 with
    // plain stores, gated sum + code 274.8 either way (284.5 with plain loads).
    const bool stream = V == 8 && T * A.H >= (int64_t)1 << 21;
    auto go = [&](auto comb) {
        constexpr int K = decltype(comb)::value;
        constexpr int S1 = V == 8 ? 1 : 0, S2 = V == 8 && K ? 2 : S1;
        const int64_t most = rows_of_launch(A.nw);
        for (A.t0 = 0; A.t0 < T; A.t0 += most) {
            const unsigned n = (unsigned)(T - A.t0 < most ? T - A.t0 : most);
            if (!stream) k_block<V, NCH, K, 0, ANY><<<n, A.nw * 64, 0, s>>>(A);
            else if (A.b.y_dtype == MOE_DT_F32) k_block<V, NCH, K, S1, ANY><<<n, A.nw * 64, 0, s>>>(A);
            else k_block<V, NCH, K, S2, ANY><<<n, A.nw * 64, 0, s>>>(A);
        }
    };
    if (A.b.k > 0) go(std::integral_constant<int, C>{});
    else go(std::integral_constant<int, 0>{});
}

}  // namespace

// vec8: every operand's rows start on 16 bytes and H is a multiple of 8.
int launch_block(const moe_block& b, int64_t T, int32_t H, bool vec8, void* stream) {
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    BlockRow A{b, 0, H, 1};
    auto waves = [&](int per) { return (H + 512 * per - 1) / (512 * per); };
    // As many threads as a row has chunks, up to 1024 (one token, H 6144: 3.2 us
    // against 4.0 with two chunks a thread; 4096 tokens from HBM, norm after and
    // before: 50 against 54).  Rows off 16 bytes go by the same chunks (norm after
    // and before, one token / 4096 tokens of 6145 bf16: 5.6 / 77 us against 42 / 224
    // element by element; 333 rows of 1003 fp32 5.0 against 6.0; 1008 takes 4.3).
    // The bits are the same in all of them.
    auto go = [&](auto any) {
        constexpr bool ANY = decltype(any)::value;
        if (waves(1) <= 16) { A.nw = waves(1); launch<8, 1, ANY>(A, T, s); }
        else if (waves(2) <= 16) { A.nw = waves(2); launch<8, 2, ANY>(A, T, s); }
        else { A.nw = waves(4); launch<8, 4, ANY>(A, T, s); }
    };
    if (vec8) go(std::false_type{});
    else if (H >= 8) go(std::true_type{});
    else launch<1, 1, false>(A, T, s);
    MOEQ_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace moeq
