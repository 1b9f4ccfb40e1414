// C ABI of what stands beside and behind a projection (head norms with rotation, token
// log probabilities, low-rank adapters): argument checks and dispatch to the launchers.
#include <cmath>
#include <cstdint>
#include <string>

#include "api_checks.h"

using namespace moeq;

namespace {

constexpr int32_t kMaxHeads = 4096;

// No two of the n1 x n2 runs of D elements, s1 and s2 apart, overlap.
bool apart(int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t D) {
    if (n1 == 1) return n2 == 1 || s2 >= D;
    if (n2 == 1) return s1 >= D;
    return (s2 >= D && s1 >= (n2 - 1) * s2 + D) || (s1 >= D && s2 >= (n1 - 1) * s1 + D);
}

int check_set(const std::string& fn, const char* name, const moe_head_set& s, const moe_heads& h,
              int64_t T) {
    const std::string of = fn + ": " + name;
    if (s.heads < 0 || s.heads > kMaxHeads)
        return fail(MOE_EINVAL, of + " must have 0 to " + std::to_string(kMaxHeads) + " heads");
    if (s.heads == 0) return MOE_OK;
    if (!s.x || !s.out) return fail(MOE_EINVAL, of + " is a null pointer");
    const uintptr_t b = (uintptr_t)dt_bytes(h.dtype);
    if (!aligned(s.x, b) || !aligned(s.out, b))
        return fail(MOE_EINVAL, of + " is not aligned to its element type");
    if (s.w && !aligned(s.w, (uintptr_t)dt_bytes(h.w_dtype)))
        return fail(MOE_EINVAL, of + "'s weights are not aligned to their element type");
    if (s.ld_t < 0 || s.ld_h < 0) return fail(MOE_EINVAL, of + "'s strides must be positive");
    if (T > 0 && !apart(T, s.ld_out_t, s.heads, s.ld_out_h, h.D))
        return fail(MOE_EINVAL, of + "'s output heads overlap");
    if (s.x == s.out && (s.ld_t != s.ld_out_t || s.ld_h != s.ld_out_h))
        return fail(MOE_EINVAL, of + " in place needs the same strides");
    return MOE_OK;
}

int check_adapters(const std::string& fn, const moe_adapters* S) {
    if (!S) return bad(fn, "set is NULL");
    if (S->n < 1 || S->n > MOE_MAX_ADAPTERS)
        return fail(MOE_EINVAL, fn + ": n must be in [1, " + std::to_string(MOE_MAX_ADAPTERS) + "]");
    if (!moe_adapter_bytes(0, S->rank, S->K, S->N)) return bad(fn, "bad rank, K or N");
    if (S->w_dtype != MOE_DT_BF16 && S->w_dtype != MOE_DT_F16)
        return fail(MOE_EUNSUPPORTED, fn + ": adapters are bf16 or fp16");
    if (!S->a || !S->b || !S->ranks || !S->scales) return bad(fn, "a pointer of the set is NULL");
    if (!aligned(S->a, 16) || !aligned(S->b, 16)) return bad(fn, "a and b must be 16-byte aligned");
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_head_norm_rope(const moe_heads* h, int64_t T, void* stream) {
    set_error("");
    const std::string fn = "moe_head_norm_rope";
    if (!h) return bad(fn, "heads is NULL");
    if (T < 0 || T >= kMaxRows) return bad(fn, "bad T");
    if (h->D < 1) return bad(fn, "bad D");
    if (h->D > MOE_HEAD_MAX_D)
        return fail(MOE_EUNSUPPORTED,
                    fn + ": D must be at most " + std::to_string(MOE_HEAD_MAX_D));
    if (!float_dt(h->dtype)) return fail(MOE_EUNSUPPORTED, fn + ": unknown element type");
    if ((h->q.w || h->k.w) && !float_dt(h->w_dtype))
        return fail(MOE_EUNSUPPORTED, fn + ": the weights have an unknown element type");
    if (!std::isfinite(h->eps) || h->eps < 0.f || !std::isfinite(h->w_offset))
        return bad(fn, "eps and w_offset must be finite and eps >= 0");
    int st = check_set(fn, "q", h->q, *h, T);
    if (!st) st = check_set(fn, "k", h->k, *h, T);
    if (st) return st;
    if (h->pos) {
        if (h->pos_bits != 32 && h->pos_bits != 64) return bad(fn, "pos_bits must be 32 or 64");
        if (!aligned(h->pos, (uintptr_t)h->pos_bits / 8)) return bad(fn, "pos is misaligned");
        if (h->R < 2 || h->R > h->D || h->R % 2) return bad(fn, "R must be even and in [2, D]");
        if (!h->table || h->table_rows < 1) return bad(fn, "pos needs a table");
        if (!aligned(h->table, 4)) return bad(fn, "table is misaligned");
    } else if (!h->q.w && !h->k.w) {
        return bad(fn, "neither weights nor positions are given");
    }
    if (T == 0 || h->q.heads + h->k.heads == 0) return MOE_OK;
    moe_heads v = *h;
    if (!v.pos) v.R = 0;
    return launch_heads(v, T, stream);
}

size_t moe_token_logprobs_workspace_bytes(int64_t T, int32_t V, int32_t top) {
    if (T < 0 || T >= kMaxRows || V < 1 || V > MOE_MAX_VOCAB || top < 0 || top > MOE_MAX_TOP)
        return 0;
    return (size_t)T * (size_t)(round_up(V, kLogprobSlice) / kLogprobSlice) *
           (16 + 8 * (size_t)top);
}

int moe_token_logprobs(const moe_logprobs* a, int64_t T, void* ws, size_t ws_bytes,
                       void* stream) {
    set_error("");
    const std::string fn = "moe_token_logprobs";
    if (!a) return bad(fn, "args is NULL");
    if (T < 0 || T >= kMaxRows) return bad(fn, "bad T");
    if (a->V < 1) return bad(fn, "bad V");
    if (a->V > MOE_MAX_VOCAB)
        return fail(MOE_EUNSUPPORTED,
                    fn + ": V must be at most " + std::to_string(MOE_MAX_VOCAB));
    if (a->top < 0 || a->top > MOE_MAX_TOP)
        return fail(MOE_EINVAL, fn + ": top must be in [0, " + std::to_string(MOE_MAX_TOP) + "]");
    if (a->m < 0 || a->m > 1024) return bad(fn, "m must be in [0, 1024]");
    if (T == 0) return MOE_OK;
    if (!a->logits) return bad(fn, "logits is NULL");
    bool vec8 = false;
    int st = check_rows(fn, "logits", a->logits, a->dtype, a->ld, a->V, vec8);
    if (st) return st;
    if (!a->ids != !a->m || !a->ids != !a->logprob)
        return bad(fn, "ids, m and logprob go together");
    if (a->ids && a->id_bits != 32 && a->id_bits != 64)
        return bad(fn, "id_bits must be 32 or 64");
    if (a->ids && !aligned(a->ids, (uintptr_t)a->id_bits / 8)) return bad(fn, "ids is misaligned");
    if (a->top ? !a->top_ids || !a->top_logprob : a->top_ids || a->top_logprob)
        return bad(fn, "top, top_ids and top_logprob go together");
    if (!a->ids && !a->entropy && !a->top) return bad(fn, "no output is given");
    const size_t need = moe_token_logprobs_workspace_bytes(T, a->V, a->top);
    if (!ws || ws_bytes < need)
        return fail(MOE_EWORKSPACE, fn + ": workspace needs " + std::to_string(need) + " bytes");
    if (!aligned(ws, kAlign)) return bad(fn, "workspace must be 256-byte aligned");
    return launch_logprobs(*a, T, ws, stream);
}

size_t moe_adapter_bytes(int which, int32_t rank, int32_t K, int32_t N) {
    if (which < 0 || which > 1 || rank < 1 || rank > MOE_MAX_RANK || K < 1 || K > kMaxDim || N < 1 ||
        N > kMaxDim)
        return 0;
    return (size_t)(which == 0 ? ad_a_bytes(rank, K) : ad_b_bytes(rank, N));
}

int moe_pack_adapter(const moe_adapters* set, int32_t slot, const void* a, int64_t lda,
                     const void* b, int64_t ldb, int32_t rank, float scale, void* stream) {
    set_error("");
    const std::string fn = "moe_pack_adapter";
    int st = check_adapters(fn, set);
    if (st) return st;
    if (slot < 0 || slot >= set->n) return bad(fn, "slot must be in [0, n)");
    if (rank < 0 || rank > set->rank) return bad(fn, "rank must be in [0, the set's rank]");
    if (!std::isfinite(scale)) return bad(fn, "scale must be finite");
    if (rank) {
        if (!a || !b) return bad(fn, "null pointer");
        if (!aligned(a, 2) || !aligned(b, 2)) return bad(fn, "a and b must be 2-byte aligned");
        if (lda < set->K || ldb < rank) return bad(fn, "a row stride is below the width");
    }
    if ((ad_a_bytes(set->rank, set->K) + ad_b_bytes(set->rank, set->N)) / 16 >=
        256 * rows_of_launch(4))
        return fail(MOE_EUNSUPPORTED, fn + ": the adapter is too large for one launch");
    return launch_pack_adapter(*set, slot, a, lda, b, ldb, rank, scale, stream);
}

size_t moe_adapter_plan_bytes(int64_t T, int32_t n) {
    if (T < 0 || T >= kMaxRows - 4096 || n < 1 || n > MOE_MAX_ADAPTERS) return 0;
    // never less for more tokens: records of 16 would need more than some of 64 do
    const int64_t some = ad_plan(T, n, 16).total, own = ad_plan(T, n).total;
    return (size_t)(some > own ? some : own) * 4;
}

int moe_adapter_plan(const int32_t* ids, int64_t T, int32_t n, void* plan, size_t plan_bytes,
                     void* stream) {
    set_error("");
    const std::string fn = "moe_adapter_plan";
    const size_t need = moe_adapter_plan_bytes(T, n);
    if (!need) return bad(fn, "bad T or n");
    if (T == 0) return MOE_OK;
    if (!ids || !plan) return bad(fn, "null pointer");
    if (!aligned(ids, 4)) return bad(fn, "ids is misaligned");
    if (!aligned(plan, 16)) return bad(fn, "plan must be 16-byte aligned");
    if (plan_bytes < need)
        return fail(MOE_EWORKSPACE, fn + ": the plan needs " + std::to_string(need) + " bytes");
    return launch_adapter_plan(ids, T, n, static_cast<int32_t*>(plan), stream);
}

size_t moe_add_adapters_workspace_bytes(const moe_adapters* set, int64_t T) {
    if (!set || !moe_adapter_plan_bytes(T, set->n) || set->rank < 1 || set->rank > MOE_MAX_RANK || set->K < 1)
        return 0;
    return align_up(add_adapters_ws_bytes(*set, T));
}

int moe_add_adapters(const moe_adapters* set, const void* x, int32_t x_dtype, int64_t ldx,
                     const float* x_scale, const void* plan, int64_t T, const void* y, int64_t ldy,
                     void* out, int64_t ldo, int32_t y_dtype, void* ws, size_t ws_bytes,
                     void* stream) {
    set_error("");
    const std::string fn = "moe_add_adapters";
    int st = check_adapters(fn, set);
    if (st) return st;
    if (!moe_adapter_plan_bytes(T, set->n)) return bad(fn, "bad T");
    if (T == 0) return MOE_OK;
    if (!x || !plan || !y || !out) return bad(fn, "null pointer");
    bool vec8 = false;
    if (x_dtype == MOE_DT_I8) {
        if (!x_scale) return bad(fn, "codes need x_scale");
        if ((st = check_codes(fn, "x", x, ldx, set->K))) return st;
    } else {
        if (x_scale) return bad(fn, "x_scale goes with codes (MOE_DT_I8) only");
        if (x_dtype != set->w_dtype)
            return fail(MOE_EUNSUPPORTED, fn + ": x must be of the adapters' type, or 8-bit codes");
        if ((st = check_rows(fn, "x", x, x_dtype, ldx, set->K, vec8))) return st;
    }
    if ((st = check_rows(fn, "y", y, y_dtype, ldy, set->N, vec8))) return st;
    if ((st = check_rows(fn, "out", out, y_dtype, ldo, set->N, vec8))) return st;
    if (y == out && ldy != ldo) return bad(fn, "in place needs the same stride");
    if (!aligned(plan, 16)) return bad(fn, "plan must be 16-byte aligned");
    const size_t need = moe_add_adapters_workspace_bytes(set, T);
    if (!ws || ws_bytes < need)
        return fail(MOE_EWORKSPACE, fn + ": workspace needs " + std::to_string(need) + " bytes");
    if (!aligned(ws, kAlign)) return bad(fn, "workspace must be 256-byte aligned");
    // the shrink's grid, at most: 16-token pieces by rank tiles by parts
    const AdPlan lay = ad_plan(T, set->n);
    if (lay.tiles * (lay.tile / 16) * ad_rank_tiles(set->rank) * kAdParts >=
        rows_of_launch(kAdWaves))
        return fail(MOE_EUNSUPPORTED, fn + ": too many tokens for one call");
    return launch_add_adapters(*set, x, x_dtype, ldx, x_scale, static_cast<const int32_t*>(plan),
                               T, y, out, y_dtype, ldy, ldo, static_cast<float*>(ws), stream);
}

}  // extern "C"
