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
// per thread), so every operand is read once and every result written once;
// the reductions (b^2, r'^2, max |n|) go through LDS.
#include "elem_dev.h"

namespace moeq {

namespace {

struct BlockRow {
    moe_block b;
    int H, nw;
};

template <int V, int NCH, bool COMB>
__global__ __launch_bounds__(1024) void k_block(BlockRow A) {
    __shared__ float red[3][16];
    const moe_block& b = A.b;
    const int64_t t = blockIdx.x;
    const int H = A.H, nt = A.nw * 64;
    float v[NCH][V];

    // ------------------------------------------------ the block's output
    if constexpr (COMB) {
        const float sg = b.y_shared && b.shared_gate ? b.shared_gate[t] : 1.f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int h = (c * nt + (int)threadIdx.x) * V;
#pragma unroll
            for (int e = 0; e < V; ++e) v[c][e] = 0.f;
            if (h >= H) continue;
            for (int j = 0; j < b.k; ++j) {
                const int64_t row = b.inv_perm[t * b.k + j];
                const float wj = b.topk_w[t * b.k + j];
                float y[V];
                load_f32<V>(b.y, b.y_dtype, row * b.ld_y + h, y);
#pragma unroll
                for (int e = 0; e < V; ++e) v[c][e] += wj * y[e];
            }
            if (b.y_shared) {
                float y[V];
                load_f32<V>(b.y_shared, b.y_shared_dtype, t * b.ld_y_shared + h, y);
#pragma unroll
                for (int e = 0; e < V; ++e) v[c][e] += sg * y[e];
            }
        }
    } else if (b.y) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int h = (c * nt + (int)threadIdx.x) * V;
            if (h < H) {
                load_f32<V>(b.y, b.y_dtype, t * b.ld_y + h, v[c]);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) v[c][e] = 0.f;
            }
        }
    }

    // ------------------------------------------------ the norm after
    const bool has_y = COMB || b.y;
    float rstd = 1.f;
    if (has_y && b.post_w) {
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int e = 0; e < V; ++e) ss += v[c][e] * v[c][e];
        ss = block_sum(ss, red[0], A.nw);
        rstd = 1.f / sqrtf(ss / (float)H + b.eps);
    }

    // ------------------------------------------------ gate, scales, residual
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int h = (c * nt + (int)threadIdx.x) * V;
        if (h >= H) {
#pragma unroll
            for (int e = 0; e < V; ++e) v[c][e] = 0.f;
            continue;
        }
        if (has_y) {
            if (b.post_w) {
                float w[V];
                load_f32<V>(b.post_w, b.w_dtype, h, w);
#pragma unroll
                for (int e = 0; e < V; ++e) v[c][e] = v[c][e] * rstd * (b.w_offset + w[e]);
            }
            if (b.gate) {
                float g[V];
                if (b.gate_ld_h) {
                    load_f32<V>(b.gate, b.gate_dtype, t * b.gate_ld_t + h, g);
                } else {
                    const float g1 = load_elem(b.gate, b.gate_dtype, t * b.gate_ld_t);
#pragma unroll
                    for (int e = 0; e < V; ++e) g[e] = g1;
                }
#pragma unroll
                for (int e = 0; e < V; ++e) v[c][e] *= g[e];
            }
#pragma unroll
            for (int e = 0; e < V; ++e) v[c][e] *= b.y_scale;
        }
        if (b.r) {
            float r[V];
            load_f32<V>(b.r, b.r_dtype, t * b.ld_r + h, r);
#pragma unroll
            for (int e = 0; e < V; ++e)
                v[c][e] = has_y ? b.r_scale * r[e] + v[c][e] : b.r_scale * r[e];
        }
        if (b.r_out) store_f32<V>(b.r_out, b.r_dtype, t * b.ld_r_out + h, v[c]);
    }
    if (!b.n_out && !b.q_out) return;

    // ------------------------------------------------ the norm before the next
    if (b.pre_w) {
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int e = 0; e < V; ++e) ss += v[c][e] * v[c][e];
        ss = block_sum(ss, red[1], A.nw);
        rstd = 1.f / sqrtf(ss / (float)H + b.eps);
    }
    uint32_t amax = 0u;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int h = (c * nt + (int)threadIdx.x) * V;
        if (h >= H) continue;
        if (b.pre_w) {
            float w[V];
            load_f32<V>(b.pre_w, b.w_dtype, h, w);
#pragma unroll
            for (int e = 0; e < V; ++e) v[c][e] = v[c][e] * rstd * (b.w_offset + w[e]);
        }
        if (b.n_out) store_f32<V>(b.n_out, b.n_dtype, t * b.ld_n + h, v[c]);
#pragma unroll
        for (int e = 0; e < V; ++e) amax = max(amax, __float_as_uint(v[c][e]) & 0x7fffffffu);
    }
    if (!b.q_out) return;

    // ------------------------------------------------ its 8-bit code
    amax = block_max(amax, reinterpret_cast<uint32_t*>(red[2]), A.nw);
    const RowCode rc = row_code(amax);
    if (threadIdx.x == 0) b.q_scale[t] = rc.scale;
    int8_t* q = b.q_out + t * b.ld_q;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int h = (c * nt + (int)threadIdx.x) * V;
        if (h >= H) continue;
        if constexpr (V == 8) {
            const uint2 u = {pack_codes4(&v[c][0], rc.mul), pack_codes4(&v[c][4], rc.mul)};
            *reinterpret_cast<uint2*>(q + h) = u;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) q[h + e] = (int8_t)code_of(v[c][e], rc.mul);
        }
    }
    const int pad = (H + 63) / 64 * 64 - H;
    if ((int)threadIdx.x < pad) q[H + threadIdx.x] = 0;
}

template <int V, int NCH>
void launch(const BlockRow& A, int64_t T, hipStream_t s) {
    if (A.b.k > 0)
        k_block<V, NCH, true><<<(unsigned)T, A.nw * 64, 0, s>>>(A);
    else
        k_block<V, NCH, false><<<(unsigned)T, A.nw * 64, 0, s>>>(A);
}

}  // namespace

// vec8: every operand's rows start on 16 bytes and H is a multiple of 8.
int launch_block(const moe_block& b, int64_t T, int32_t H, bool vec8, void* stream) {
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const int V = vec8 ? 8 : 1;
    const int nch = (H + V - 1) / V;
    BlockRow A{b, H, 1};
    auto waves = [&](int per) { return (nch + 64 * per - 1) / (64 * per); };
    if (vec8) {
        if (waves(1) <= 16) { A.nw = waves(1); launch<8, 1>(A, T, s); }
        else if (waves(2) <= 16) { A.nw = waves(2); launch<8, 2>(A, T, s); }
        else { A.nw = waves(4); launch<8, 4>(A, T, s); }
    } else {
        if (waves(8) <= 16) { A.nw = waves(8); launch<1, 8>(A, T, s); }
        else { A.nw = waves(32); launch<1, 32>(A, T, s); }
    }
    MOEQ_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace moeq
