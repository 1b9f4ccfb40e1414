// C ABI of the block norms and the 8-bit integer products: argument checks,
// workspace layout and dispatch to the HIP launchers.
#include <cmath>
#include <cstdint>
#include <string>

#include "api_checks.h"

using namespace moeq;

namespace {

constexpr int32_t kMaxI8K = 131071;   // 2^31 / (128 * 128): int32 sums cannot wrap

// The products' tiles are 128 rows by 256 channels wherever they are many, and
// no smaller than 32 rows for up to 64 rows of each expert: the workgroups of a
// pass, 256 threads each, are one launch of less than 2^32 threads.
int check_tiles(const std::string& fn, int64_t rows, int64_t E, int64_t N) {
    const int64_t bm = rows > 64 * (int64_t)MOE_MAX_E ? 128 : 32;
    if ((rows / bm + E + 1) * (N / 256 + 1) >= rows_of_launch(4) - 64)
        return fail(MOE_EUNSUPPORTED, fn + ": too many rows and channels for one call");
    return MOE_OK;
}

// x as the product calls take it: codes with a scale per row, or rows of a
// float type that the call quantises into its workspace.
int check_x(const std::string& fn, const void* x, int dt, int64_t ldx, const float* x_scale,
            int64_t K, bool& vec8) {
    if (!x) return bad(fn, "x is NULL");
    if (dt == MOE_DT_I8) {
        if (!x_scale) return bad(fn, "codes need x_scale");
        return check_codes(fn, "x", x, ldx, K);
    }
    if (x_scale) return bad(fn, "x_scale goes with codes (MOE_DT_I8) only");
    vec8 = K % 8 == 0;
    return check_rows(fn, "x", x, dt, ldx, K, vec8);
}

// Codes and scales of x in a workspace: [T, round_up(K, 64)] then [T].
size_t codes_ws(int64_t T, int32_t K) {
    return align_up((size_t)T * (size_t)round_up(K, kI8TileK)) + align_up((size_t)T * 4);
}

// The rows of pass p: codes as they are; float rows handed to the kernel that
// codes them itself, or coded into ws (codes_ws bytes) first.  T, k are the
// batch's; n rows are here.
int take_rows(I8Pass& p, const void* x, int dt, int64_t ldx, const float* x_scale, int64_t n,
              bool vec8, uint8_t* ws, void* stream) {
    p.x = nullptr;
    if (dt == MOE_DT_I8) {
        p.q = static_cast<const int8_t*>(x);
        p.ldq = ldx;
        p.qscale = x_scale;
        return MOE_OK;
    }
    if (i8_codes_itself(p.T, p.K, p.offsets != nullptr)) {
        p.x = x;
        p.ldx = ldx;
        p.x_dtype = dt;
        p.x_vec8 = vec8;
        return MOE_OK;
    }
    const int64_t ldq = round_up(p.K, kI8TileK);
    int8_t* q = reinterpret_cast<int8_t*>(ws);
    float* scale = reinterpret_cast<float*>(ws + align_up((size_t)n * (size_t)ldq));
    p.q = q;
    p.ldq = ldq;
    p.qscale = scale;
    return launch_quantize_i8(x, dt, ldx, n, p.K, q, ldq, scale, vec8, stream);
}

int check_linear(const std::string& fn, const moe_i8_linear* L) {
    if (!L) return bad(fn, "linear is NULL");
    if (L->N < 1 || L->K < 1 || L->N > kMaxDim) return bad(fn, "bad N or K");
    if (L->K > kMaxI8K)
        return fail(MOE_EUNSUPPORTED, fn + ": K must be at most " + std::to_string(kMaxI8K));
    if (!L->w || !L->w_scale) return bad(fn, "weights or scales are NULL");
    if (!aligned(L->w, 16)) return bad(fn, "weights must be 16-byte aligned");
    return MOE_OK;
}

int check_i8_layer(const std::string& fn, const moe_i8_layer* L) {
    if (!L) return bad(fn, "layer is NULL");
    if (L->E < 1 || L->E > MOE_MAX_E) return bad(fn, "bad E");
    if (L->H < 1 || L->I < 1) return bad(fn, "bad H or I");
    if (L->H > kMaxI8K || L->I > kMaxI8K)
        return fail(MOE_EUNSUPPORTED,
                    fn + ": H and I must be at most " + std::to_string(kMaxI8K));
    if (!L->w13 || !L->w2 || !L->w13_scale || !L->w2_scale)
        return bad(fn, "weights or scales are NULL");
    if (!aligned(L->w13, 16) || !aligned(L->w2, 16) || L->w13_stride % 16 || L->w2_stride % 16)
        return bad(fn, "weights must be 16-byte aligned");
    if (L->w13_stride < (int64_t)moe_i8_record_bytes(0, L->H, L->I) ||
        L->w2_stride < (int64_t)moe_i8_record_bytes(1, L->H, L->I))
        return bad(fn, "record stride below moe_i8_record_bytes()");
    return MOE_OK;
}

// x codes | h [rows, I] fp32 | h codes
struct FfnWs {
    size_t h, hq, total;
};

FfnWs ffn_i8_ws(const moe_i8_layer* L, int64_t T, int32_t k) {
    FfnWs w;
    const size_t rows = (size_t)T * (size_t)k;
    w.h = codes_ws(T, L->H);
    w.hq = w.h + align_up(rows * (size_t)L->I * 4);
    w.total = w.hq + codes_ws((int64_t)rows, L->I);
    return w;
}

// Both FFN calls: the routed experts (offsets != NULL) or the one expert of
// every token.
int run_ffn_i8(const std::string& fn, const moe_i8_layer* L, const void* x, int32_t x_dtype,
               int64_t ldx, const float* x_scale, const int32_t* perm_src, const int32_t* offsets,
               int64_t T, int32_t k, void* y, int32_t y_dtype, void* ws, size_t ws_bytes,
               void* stream) {
    if (!float_dt(y_dtype)) return fail(MOE_EUNSUPPORTED, fn + ": unknown output type");
    if (!aligned(y, (uintptr_t)dt_bytes(y_dtype))) return bad(fn, "the output is misaligned");
    bool vec8 = false;
    int st = check_x(fn, x, x_dtype, ldx, x_scale, L->H, vec8);
    if (st) return st;
    st = check_tiles(fn, T * k, L->E, 2 * (int64_t)(L->H > L->I ? L->H : L->I));
    if (st) return st;
    const FfnWs lay = ffn_i8_ws(L, T, k);
    if (!ws || ws_bytes < lay.total)
        return fail(MOE_EWORKSPACE,
                    fn + ": workspace needs " + std::to_string(lay.total) + " bytes");
    if (!aligned(ws, kAlign)) return bad(fn, "workspace must be 256-byte aligned");
    uint8_t* w = static_cast<uint8_t*>(ws);
    const int64_t rows = T * k;
    float* h = reinterpret_cast<float*>(w + lay.h);
    I8Pass p{};
    p.w = static_cast<const uint8_t*>(L->w13);
    p.w_stride = L->w13_stride;
    p.wscale = L->w13_scale;
    p.wscale_stride = 2 * (int64_t)L->I;
    p.offsets = offsets;
    p.perm_src = perm_src;
    p.T = T;
    p.E = L->E;
    p.k = k;
    p.N = L->I;
    p.K = L->H;
    p.out = h;
    p.ld_out = L->I;
    p.out_dtype = MOE_DT_F32;
    st = take_rows(p, x, x_dtype, ldx, x_scale, T, vec8, w, stream);
    if (st) return st;
    st = launch_i8(p, true, stream);
    if (st) return st;
    p.w = static_cast<const uint8_t*>(L->w2);
    p.w_stride = L->w2_stride;
    p.wscale = L->w2_scale;
    p.wscale_stride = L->H;
    p.perm_src = nullptr;
    p.N = L->H;
    p.K = L->I;
    p.out = y;
    p.ld_out = L->H;
    p.out_dtype = y_dtype;
    st = take_rows(p, h, MOE_DT_F32, L->I, nullptr, rows, L->I % 8 == 0, w + lay.hq, stream);
    if (st) return st;
    return launch_i8(p, false, stream);
}

}  // namespace

extern "C" {

int moe_block_norm(const moe_block* b, int64_t T, int32_t H, void* stream) {
    set_error("");
    const std::string fn = "moe_block_norm";
    if (!b) return bad(fn, "block is NULL");
    if (T < 0 || T >= kMaxRows) return bad(fn, "bad T");
    if (H < 1) return bad(fn, "bad H");
    if (H > MOE_BLOCK_MAX_H)
        return fail(MOE_EUNSUPPORTED,
                    fn + ": H must be at most " + std::to_string(MOE_BLOCK_MAX_H));
    if (b->k < 0 || b->k > MOE_MAX_K) return bad(fn, "k must be in [0, 16]");
    if (T * (int64_t)(b->k > 0 ? b->k : 1) >= kMaxRows) return bad(fn, "T*k too large");
    if (!std::isfinite(b->y_scale) || !std::isfinite(b->r_scale) || !std::isfinite(b->w_offset) ||
        !std::isfinite(b->eps) || b->eps < 0.f)
        return bad(fn, "scales, w_offset and eps must be finite and eps >= 0");
    if (T == 0) return MOE_OK;
    if (!b->y && !b->r) return bad(fn, "neither y nor r is given");
    if (!b->y && (b->k || b->y_shared || b->post_w || b->gate))
        return bad(fn, "k, y_shared, post_w and gate need y");
    if (b->k ? !b->inv_perm || !b->topk_w : b->inv_perm || b->topk_w || b->y_shared)
        return bad(fn, "inv_perm and topk_w go with k > 0, y_shared only with them");
    if (b->shared_gate && !b->y_shared) return bad(fn, "shared_gate needs y_shared");
    if (!b->r_out && !b->n_out && !b->q_out) return bad(fn, "no output is given");
    if (!b->q_out != !b->q_scale) return bad(fn, "q_out and q_scale go together");
    bool vec8 = H % 8 == 0;
    int st = MOE_OK;
    if (b->y && (st = check_rows(fn, "y", b->y, b->y_dtype, b->ld_y, H, vec8))) return st;
    if (b->y_shared && (st = check_rows(fn, "y_shared", b->y_shared, b->y_shared_dtype,
                                        b->ld_y_shared, H, vec8)))
        return st;
    if (b->r && (st = check_rows(fn, "r", b->r, b->r_dtype, b->ld_r, H, vec8))) return st;
    if (b->r_out && (st = check_rows(fn, "r_out", b->r_out, b->r_dtype, b->ld_r_out, H, vec8)))
        return st;
    if (b->n_out && (st = check_rows(fn, "n_out", b->n_out, b->n_dtype, b->ld_n, H, vec8)))
        return st;
    if (b->post_w && (st = check_rows(fn, "post_w", b->post_w, b->w_dtype, H, H, vec8))) return st;
    if (b->pre_w && (st = check_rows(fn, "pre_w", b->pre_w, b->w_dtype, H, H, vec8))) return st;
    if (b->gate) {
        if (b->gate_ld_h != 0 && b->gate_ld_h != 1) return bad(fn, "gate_ld_h must be 0 or 1");
        if (b->gate_ld_t < 0) return bad(fn, "gate_ld_t < 0");
        bool v = vec8;
        // a gate of one value per token, or one row for every token, has no row stride to check
        const int64_t ld = b->gate_ld_h && b->gate_ld_t ? b->gate_ld_t : H;
        if ((st = check_rows(fn, "gate", b->gate, b->gate_dtype, ld, H, v))) return st;
        if (b->gate_ld_h) vec8 = v;
    }
    if (b->q_out && (st = check_codes(fn, "q_out", b->q_out, b->ld_q, H))) return st;
    return launch_block(*b, T, H, vec8, stream);
}

int moe_quantize_i8(const void* x, int32_t x_dtype, int64_t ldx, int64_t T, int32_t K, int8_t* q,
                    int64_t ldq, float* scale, void* stream) {
    set_error("");
    const std::string fn = "moe_quantize_i8";
    if (T < 0 || T >= kMaxRows) return bad(fn, "bad T");
    if (K < 1 || K > kMaxDim) return bad(fn, "bad K");
    if (T == 0) return MOE_OK;
    if (!x || !q || !scale) return bad(fn, "null pointer");
    bool vec8 = K % 8 == 0;
    int st = check_rows(fn, "x", x, x_dtype, ldx, K, vec8);
    if (st) return st;
    st = check_codes(fn, "q", q, ldq, K);
    if (st) return st;
    return launch_quantize_i8(x, x_dtype, ldx, T, K, q, ldq, scale, vec8, stream);
}

size_t moe_i8_matrix_bytes(int32_t N, int32_t K) {
    if (N < 1 || K < 1 || N > kMaxDim || K > kMaxI8K) return 0;
    return (size_t)i8_matrix_bytes(N, K);
}

size_t moe_i8_record_bytes(int which, int32_t H, int32_t I) {
    if (which < 0 || which > 1 || H < 1 || I < 1 || H > kMaxI8K || I > kMaxI8K) return 0;
    return (size_t)(which == 0 ? 2 * i8_matrix_bytes(I, H) : i8_matrix_bytes(H, I));
}

int moe_pack_i8(const int8_t* codes, int64_t ld, int32_t N, int32_t K, void* packed,
                void* stream) {
    set_error("");
    const std::string fn = "moe_pack_i8";
    if (moe_i8_matrix_bytes(N, K) == 0) return bad(fn, "bad N or K");
    if (moe_i8_matrix_bytes(N, K) / kI8TileBytes >= 4 * (uint64_t)rows_of_launch(4))
        return fail(MOE_EUNSUPPORTED, fn + ": the matrix is too large for one launch");
    if (ld < K) return bad(fn, "the row stride is below K");
    if (!codes || !packed) return bad(fn, "null pointer");
    if (!aligned(packed, 16)) return bad(fn, "packed must be 16-byte aligned");
    return launch_pack_i8(codes, ld, N, K, 0, 1, packed, stream);
}

int moe_pack_i8_expert(const int8_t* gate, const int8_t* up, const int8_t* down, int32_t H,
                       int32_t I, void* w13_rec, void* w2_rec, void* stream) {
    set_error("");
    const std::string fn = "moe_pack_i8_expert";
    if (moe_i8_record_bytes(0, H, I) == 0) return bad(fn, "bad H or I");
    if (!gate || !up || !down || !w13_rec || !w2_rec) return bad(fn, "null pointer");
    if (!aligned(w13_rec, 16) || !aligned(w2_rec, 16))
        return bad(fn, "records must be 16-byte aligned");
    int st = launch_pack_i8(gate, H, I, H, 0, 2, w13_rec, stream);
    if (!st) st = launch_pack_i8(up, H, I, H, 1, 2, w13_rec, stream);
    if (!st) st = launch_pack_i8(down, I, H, I, 0, 1, w2_rec, stream);
    return st;
}

size_t moe_linear_i8_workspace_bytes(const moe_i8_linear* linear, int64_t T) {
    if (!linear || T < 0 || linear->N < 1 || linear->K < 1) return 0;
    return codes_ws(T, linear->K);
}

int moe_linear_i8(const moe_i8_linear* linear, const void* x, int32_t x_dtype, int64_t ldx,
                  const float* x_scale, int64_t T, void* out, int32_t out_dtype, int64_t ldo,
                  void* ws, size_t ws_bytes, void* stream) {
    set_error("");
    const std::string fn = "moe_linear_i8";
    int st = check_linear(fn, linear);
    if (st) return st;
    if (T < 0 || T >= kMaxRows) return bad(fn, "bad T");
    if (!float_dt(out_dtype)) return fail(MOE_EUNSUPPORTED, fn + ": unknown output type");
    if (T == 0) return MOE_OK;
    if (!out) return bad(fn, "out is NULL");
    if (!aligned(out, (uintptr_t)dt_bytes(out_dtype))) return bad(fn, "out is misaligned");
    if (ldo < linear->N) return bad(fn, "the row stride of out is below N");
    bool vec8 = false;
    st = check_x(fn, x, x_dtype, ldx, x_scale, linear->K, vec8);
    if (st) return st;
    st = check_tiles(fn, T, 1, linear->N);
    if (st) return st;
    if (x_dtype != MOE_DT_I8) {
        const size_t need = codes_ws(T, linear->K);
        if (!ws || ws_bytes < need)
            return fail(MOE_EWORKSPACE, fn + ": workspace needs " + std::to_string(need) + " bytes");
        if (!aligned(ws, kAlign)) return bad(fn, "workspace must be 256-byte aligned");
    }
    I8Pass p{};
    p.w = static_cast<const uint8_t*>(linear->w);
    p.wscale = linear->w_scale;
    p.bias = linear->bias;
    p.T = T;
    p.E = p.k = 1;
    p.N = linear->N;
    p.K = linear->K;
    p.out = out;
    p.ld_out = ldo;
    p.out_dtype = out_dtype;
    st = take_rows(p, x, x_dtype, ldx, x_scale, T, vec8, static_cast<uint8_t*>(ws), stream);
    if (st) return st;
    return launch_i8(p, false, stream);
}

size_t moe_expert_ffn_i8_workspace_bytes(const moe_i8_layer* layer, int64_t T, int32_t k) {
    if (!layer || T < 0 || k < 1 || layer->H < 1 || layer->I < 1) return 0;
    return ffn_i8_ws(layer, T, k).total;
}

int moe_expert_ffn_i8(const moe_i8_layer* layer, const void* x, int32_t x_dtype, int64_t ldx,
                      const float* x_scale, const int32_t* perm_src, const int32_t* offsets,
                      int64_t T, int32_t k, void* y_perm, int32_t y_dtype, void* ws,
                      size_t ws_bytes, void* stream) {
    set_error("");
    const std::string fn = "moe_expert_ffn_i8";
    int st = check_i8_layer(fn, layer);
    if (st) return st;
    if (T < 0) return bad(fn, "T < 0");
    if (k < 1 || k > layer->E || k > MOE_MAX_K) return bad(fn, "k must be in [1, min(E, 16)]");
    if (T >= kMaxRows / k) return bad(fn, "T*k too large");
    if (T == 0) return MOE_OK;
    if (!perm_src || !offsets || !y_perm) return bad(fn, "null pointer");
    return run_ffn_i8(fn, layer, x, x_dtype, ldx, x_scale, perm_src, offsets, T, k, y_perm,
                      y_dtype, ws, ws_bytes, stream);
}

int moe_shared_ffn_i8(const moe_i8_layer* shared, const void* x, int32_t x_dtype, int64_t ldx,
                      const float* x_scale, int64_t T, void* y_shared, int32_t y_dtype, void* ws,
                      size_t ws_bytes, void* stream) {
    set_error("");
    const std::string fn = "moe_shared_ffn_i8";
    int st = check_i8_layer(fn, shared);
    if (st) return st;
    if (shared->E != 1) return bad(fn, "the shared layer must have E == 1");
    if (T < 0 || T >= kMaxRows) return bad(fn, "bad T");
    if (T == 0) return MOE_OK;
    if (!y_shared) return bad(fn, "null pointer");
    return run_ffn_i8(fn, shared, x, x_dtype, ldx, x_scale, nullptr, nullptr, T, 1, y_shared,
                      y_dtype, ws, ws_bytes, stream);
}

}  // extern "C"
