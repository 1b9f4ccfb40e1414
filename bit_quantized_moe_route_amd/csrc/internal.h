// Internal declarations shared by the library's translation units.
#pragma once

#include <cstddef>
#include <cstdint>
#include <string>

#include "moeq.h"

namespace moeq {

// Per-thread detail of the last rejected call (read by moe_last_error).
void set_error(const std::string& msg);
int fail(int status, const std::string& msg);

// Record geometry ------------------------------------------------------------
//
// NVFP4 tile: 16 rows x 128 inputs = 1024 code bytes + 128 scale bytes.
//   code bytes: lane L (0..63) owns bytes [16L, 16L+16): row (L & 15),
//     inputs kb*128 + (L >> 4)*32 + [0, 32), canonical nibble order.
//   scale bytes: lane L owns bytes 1024 + [2L, 2L+2): the two E4M3 scales of
//     those 32 inputs.
// VQ tile: 16 rows x 256 inputs = 1024 code bytes.
//   lane L owns bytes [16L, 16L+16) = 8 uint16 codes: row (L & 15), groups
//     covering inputs kb*256 + (L >> 4)*64 + 8s + [0, 8), s = 0..7.
// VQ8 tile (m = 1, 2 or 3 uint8 codes per group): 16 rows x 256 inputs =
//   512 m code bytes; lane L owns bytes [8mL, 8mL + 8m): row (L & 15), the
//   groups of inputs kb*256 + (L >> 4)*64 + 8s + [0, 8), s = 0..7, each group's
//   m codes consecutive (code j of group s at byte m*s + j).
// BF16 tile: 16 rows x 128 inputs = 4096 bytes in 4 slices of 1024: slice j,
//   lane L owns bytes [1024j + 16L, +16) = 8 bf16 weights of row (L & 15),
//   inputs kb*128 + (L >> 4)*32 + 8j + [0, 8) (so one 16-byte load per lane
//   reads a contiguous 1 KB slice).
// A record is a sequence of row groups of 16 rows, each a sequence of tiles
// along the input dimension (padded with zero codes/scales).  Gate/up
// records interleave row groups: group 2j = gate rows 16j.., 2j+1 = up rows.
// VQ and VQ8 records end with the fp16 per-row scales (gate, up / down),
// padded to 256 bytes.
constexpr int kNvTileK = 128;
constexpr int kNvTileBytes = 1152;
constexpr int kNvScaleOff = 1024;
constexpr int kVqTileK = 256;
constexpr int kVqTileBytes = 1024;
constexpr int kVq8TileK = 256;
constexpr int kVq8TileBytesPerCode = 512;   // times m
constexpr int kBf16TileK = 128;
constexpr int kBf16TileBytes = 4096;
// 8-bit integer matrices (moe_i8_linear, moe_i8_layer): row groups of 16 rows
//   x tiles of 64 inputs = 1024 code bytes; lane L owns bytes [16L, 16L+16):
//   row (L & 15), inputs kt*64 + (L >> 4)*16 + [0, 16), padded with zero codes
//   to an even number of tiles.  Gate/up matrices interleave row groups as above.
constexpr int kI8TileK = 64;
constexpr int kI8TileBytes = 1024;

inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

inline int64_t nv_tiles_k(int32_t kin) { return round_up(kin, kNvTileK) / kNvTileK; }
inline int64_t vq_tiles_k(int32_t kin) { return round_up(kin, kVqTileK) / kVqTileK; }

inline int64_t nv_matrix_bytes(int32_t n, int32_t kin) {
    return (int64_t)(n / 16) * nv_tiles_k(kin) * kNvTileBytes;
}
inline int64_t vq_codes_bytes(int32_t n, int32_t kin) {
    return (int64_t)(n / 16) * vq_tiles_k(kin) * kVqTileBytes;
}
inline int64_t vq8_codes_bytes(int32_t n, int32_t kin, int32_t m) {
    return (int64_t)(n / 16) * vq_tiles_k(kin) * kVq8TileBytesPerCode * m;
}
// NVFP4 record bytes (which = 0: gate/up, 1: down); also the offset of the
// residual plane inside a MOE_FMT_NVFP4R record.
inline int64_t nv_record_bytes(int which, int32_t H, int32_t I) {
    return which == 0 ? round_up(nv_matrix_bytes(2 * I, H), 256)
                      : round_up(nv_matrix_bytes(H, I), 256);
}
constexpr int64_t i8_tiles_k(int32_t kin) {
    return ((int64_t)kin + 2 * kI8TileK - 1) / (2 * kI8TileK) * 2;
}
inline int64_t i8_matrix_bytes(int32_t n, int32_t kin) {
    return round_up(n, 16) / 16 * i8_tiles_k(kin) * kI8TileBytes;
}
inline int64_t bf16_tiles_k(int32_t kin) { return round_up(kin, kBf16TileK) / kBf16TileK; }
inline int64_t bf16_matrix_bytes(int32_t n, int32_t kin) {
    return (int64_t)(n / 16) * bf16_tiles_k(kin) * kBf16TileBytes;
}

// Launchers (device code lives in the .hip files) ----------------------------
constexpr int kNumFmt = MOE_FMT_MAX + 1;   // format tags 1 .. MOE_FMT_MAX
// Small-codebook VQ at the layer's rate (MOE_FMT_VQ8) or an explicit one.
inline bool is_vq8(int fmt) {
    return fmt == MOE_FMT_VQ8 || (fmt >= MOE_FMT_VQ8_M1 && fmt <= MOE_FMT_VQ8_M3);
}
// Codes per 8-weight group of a small-codebook VQ format.
inline int vq8_rate(int fmt, int layer_vq8_m) {
    return fmt == MOE_FMT_VQ8 ? layer_vq8_m : fmt - MOE_FMT_VQ8_M1 + 1;
}
struct LayerView {
    int32_t E, H, I;
    int32_t vq8_m;
    const int32_t* rec;
    const uint8_t* pool13[kNumFmt];   // indexed by format tag
    const uint8_t* pool2[kNumFmt];
    int64_t stride13[kNumFmt];
    int64_t stride2[kNumFmt];
    const uint8_t* cb[3];       // VQ codebooks gate, up, down
    int64_t cb_stride;
    const uint8_t* cb8[3];      // VQ8 codebooks gate, up, down: [m][256][8] fp16
    int64_t res13, res2;        // MOE_FMT_NVFP4R: residual plane offset in a record
    float res_scale;            // ... and its decode factor 2^-nvfp4r_shift
    const uint8_t* rot;         // rotation sign bits per expert (NULL: not rotated)
    int64_t rot_stride;         // bytes per expert: (2H + 3I) / 8
    int32_t rot_in2;            // Hadamard block of the down input: 128 or 512
};

int launch_route_topk(const float* logits, int64_t T, int32_t E, int32_t k,
                      int32_t* ids, float* w, void* stream);
int launch_permute(const int32_t* ids, int64_t T, int32_t k, int32_t E,
                   int32_t* counts, int32_t* offsets, int32_t* perm_src,
                   int32_t* inv_perm, void* ws, void* stream);
size_t permute_ws_bytes(int64_t T, int32_t k, int32_t E);
// As many or more, and never fewer for more tokens.
size_t permute_ws_most_bytes(int64_t T, int32_t k, int32_t E);
bool route_permute_fused_ok(int64_t T, int32_t k);
int launch_route_permute(const float* logits, int64_t T, int32_t E, int32_t k, int32_t* ids,
                         float* w, int32_t* counts, int32_t* offsets, int32_t* perm_src,
                         int32_t* inv_perm, void* stream);
int launch_combine(const float* y_perm, const int32_t* inv_perm, const float* w,
                   const float* y_shared, int64_t T, int32_t k, int32_t H, float* out,
                   void* stream);
// A rotated layer: the down outputs y' (not yet rotated back) rotated back
// per slot with its expert's down-output signs and combined as launch_combine
// does, the same bits as launch_rot_out followed by launch_combine
// (inv_perm NULL: slot (t, j) is row t*k + j).
int launch_combine_rot(const LayerView& L, const float* y_perm, const int32_t* inv_perm,
                       const int32_t* ids, const float* w, const float* y_shared, int64_t T,
                       int32_t k, float* out, void* stream);
int launch_x_to_f16(const uint16_t* x, int64_t n, uint16_t* x16, void* stream);
// gu != NULL (gate/up of a rotated layer): x is the fp16 rotated rows
// [T*k, H] in permuted order, and the raw fp32 products g | u go to
// gu [T*k, 2I] instead of h.
int launch_ffn_decode(const LayerView& L, int fmt, int n_fmt, const uint16_t* x_bf16,
                      const int32_t* perm_src, const int32_t* offsets, int64_t T,
                      int32_t k, uint16_t* h16, float* y_perm, int phase,
                      void* stream, float* gu = nullptr);
// A mixed layer of NVFP4 and one VQ form (decode batches): both formats'
// gate/up (phase 0) or down (phase 1) work in one launch, when both pick the
// same input split (ffn_decode_pair_ok); the same bits as the two launches.
bool ffn_decode_pair_ok(const LayerView& L, int fmt1, int n1, int fmt2, int n2, int64_t T,
                        int32_t k);
int launch_ffn_decode_pair(const LayerView& L, int fmt1, int n1, int fmt2, int n2,
                           const uint16_t* x_bf16, const int32_t* perm_src,
                           const int32_t* offsets, int64_t T, int32_t k, uint16_t* h16,
                           float* y_perm, int phase, void* stream);
// The one expert of a shared-expert layer through the identity map (rows
// 0 .. T-1 are tokens 0 .. T-1): phase 0 writes fp32 partial g | u to part
// (shared_part_bytes) and then h, phase 1 writes y [T, H].
#ifndef MOEQ_SH_TARGET
#define MOEQ_SH_TARGET 512
#endif
constexpr int kSharedMaxSplit = 16;                  // workgroups splitting the gate/up inputs
constexpr int kSharedTargetBlocks = MOEQ_SH_TARGET;  // gate/up workgroups aimed for
// Bytes of the fp32 partial sums the decode path of a one-expert layer of
// format fmt writes for T tokens: nsplit x T x 2I x 4 with the split that
// launch_shared_decode takes; 0 where the grouped GEMM runs instead.
size_t shared_part_bytes(int fmt, int64_t T, int32_t H, int32_t I);
int launch_shared_decode(const LayerView& L, int fmt, const uint16_t* x_bf16, int64_t T,
                         uint16_t* h16, float* part, float* y, int phase, void* stream);
// Experts at T >= kPrefillMinTokens use the grouped-GEMM kernels, every
// format for routed layers; the identity map of a one-expert layer
// (perm_src == offsets == NULL) only for NVFP4 (one or two planes) and BF16.
constexpr int64_t kPrefillMinTokens = 128;
inline bool prefill_fmt(int fmt, bool identity) {
    return !identity || fmt == MOE_FMT_NVFP4 || fmt == MOE_FMT_BF16 || fmt == MOE_FMT_NVFP4R;
}
int launch_ffn_prefill(const LayerView& L, int fmt, int n_fmt, const uint16_t* x16,
                       const int32_t* perm_src, const int32_t* offsets, int64_t T, int32_t k,
                       uint16_t* h16, float* y_perm, int phase, void* stream,
                       float* gu = nullptr);
// Rotated layers: x' = rotated rows of x per assignment (fp16 [T*k, H]);
// h' from the raw gate/up products gu (fp16 [rows, I]); y rotated back in
// place (fp32 [rows, H]).
int launch_rot_in(const LayerView& L, const uint16_t* x_bf16, const int32_t* perm_src,
                  const int32_t* offsets, int64_t T, int32_t k, uint16_t* xrot, void* stream);
// row_ids != NULL: rows in assignment order, row r of expert row_ids[r]
// (offsets unused).
int launch_rot_mid(const LayerView& L, const float* gu, const int32_t* offsets, int64_t rows,
                   uint16_t* h16, void* stream, const int32_t* row_ids = nullptr);
int launch_rot_out(const LayerView& L, float* y, const int32_t* offsets, int64_t rows,
                   void* stream);
// The small-batch fused layer (single-format layers, E <= 256, k <= 8,
// T*k <= kSmallFusedAssign): gate/up with the routing inside (topk_ids /
// topk_w written, h16 [T*k, I] in token order), then down + gated combine
// (+ y_shared) into out [T, H].  A rotated layer (H <= kSmallRotMaxH) takes
// four launches and after h16 (rounded up to 256 bytes) the raw products
// [T*k, 2I] fp32 and then y' [T*k, H] fp32 (small_rot_ws_bytes in all).
#ifndef MOEQ_SMALL_ASSIGN
#define MOEQ_SMALL_ASSIGN 16
#endif
constexpr int64_t kSmallFusedAssign = MOEQ_SMALL_ASSIGN;
constexpr int32_t kSmallRotMaxH = 12288;   // the rotated row in LDS: 2H bytes
inline size_t small_rot_ws_bytes(int64_t T, int32_t k, int32_t H, int32_t I) {
    const int64_t tk = T * k;
    return (size_t)(round_up(tk * I, 128) * 2 + round_up(tk * 2 * I, 64) * 4 + tk * H * 4);
}
int launch_layer_small(const LayerView& L, int fmt, const uint16_t* x_bf16, const float* logits,
                       int64_t T, int32_t k, int32_t* topk_ids, float* topk_w, uint16_t* h16,
                       const float* y_shared, float* out, void* stream);
// The same with a BF16 shared expert SL (E == 1, same H): out = routed sum +
// the shared FFN; sh_h16 [T, SL.I] fp16 and sh_part (shared_part_bytes) are
// its workspace.
int launch_layer_small_shared(const LayerView& L, int fmt, const LayerView& SL,
                              const uint16_t* x_bf16, const float* logits, int64_t T, int32_t k,
                              int32_t* topk_ids, float* topk_w, uint16_t* h16, uint16_t* sh_h16,
                              float* sh_part, float* out, void* stream);
int launch_dequant(const LayerView& L, int fmt, int32_t rec_index, int32_t proj,
                   float* out, void* stream);
// A launch holds less than 2^32 threads: the most workgroups of nw waves in one.
inline int64_t rows_of_launch(int nw) { return (((int64_t)1 << 32) - 1) / (64 * nw); }
// Block norms (vec8: H % 8 == 0 and every row of every operand 16-byte aligned).
int launch_block(const moe_block& b, int64_t T, int32_t H, bool vec8, void* stream);
// Rows to 8-bit codes with a scale each; codes padded with zeros to a multiple
// of 64 (vec8: K % 8 == 0, x rows 16-byte and q rows 8-byte aligned).
int launch_quantize_i8(const void* x, int dt, int64_t ldx, int64_t T, int32_t K, int8_t* q,
                       int64_t ldq, float* scale, bool vec8, void* stream);
// Row-major codes into 8-bit tiles, row group g to group g0 + g * step.
int launch_pack_i8(const int8_t* codes, int64_t ld, int32_t N, int32_t K, int g0, int step,
                   void* packed, void* stream);
// One product pass of the 8-bit kernels, over the rows of q.
//   pair = true:  groups interleave gate and up rows; h[row] = silu(g) * u
//                 (fp32, rows ld_out apart), N = I channels;
//   pair = false: out[row] = scale * wscale * sum (+ bias), N channels.
// offsets == NULL: one matrix, output row r is q row r, rows r < T.
// Otherwise output row r (in expert e's offsets range) reads q row
// perm_src[r] / k, or q row r if perm_src is NULL.
struct I8Pass {
    const uint8_t* w;
    int64_t w_stride;            // bytes per expert
    const float* wscale;
    int64_t wscale_stride;       // elements per expert
    const float* bias;
    const int8_t* q;
    int64_t ldq;
    const float* qscale;
    const void* x;               // != NULL: uncoded rows of x_dtype, ldx apart, in
    int64_t ldx;                 // place of q, which the kernel codes itself
    int32_t x_dtype;             // (i8_codes_itself)
    bool x_vec8;                 // K % 8 == 0 and rows 16-byte aligned
    const int32_t* offsets;
    const int32_t* perm_src;
    int64_t T;
    int32_t E, k, N, K;
    void* out;
    int64_t ld_out;
    int32_t out_dtype;
};
// Whether the pass takes uncoded rows: one matrix, few rows, and their codes
// fit a workgroup's LDS.
bool i8_codes_itself(int64_t T, int32_t K, bool routed);
int launch_i8(const I8Pass& p, bool pair, void* stream);
int launch_gemm_i8(const I8Pass& p, bool pair, void* stream);
// Norm and rotation of query and key heads.
int launch_heads(const moe_heads& h, int64_t T, void* stream);
// Log probabilities of rows of logits: slices of a row, at most kLogprobSlices of
// them; ws: 16 + 8 top bytes a slice.
constexpr int kLogprobSlice = 16384, kLogprobSlices = 64;
int launch_logprobs(const moe_logprobs& P, int64_t T, void* ws, void* stream);
// Low-rank adapters.  A's tiles: 16 ranks x 32 inputs, 1 KB in the order of the
// matrix instruction's operand (lane L: rank L & 15, inputs (L >> 4) * 8 + 0..7), by
// adapter, rank tile, input tile; the inputs padded with zeros to whole chains.
// B's: 64 channels x 16 ranks, 2 KB in two halves (lane L: ranks (L >> 4) * 4 + 0..3 of two
// channels), by adapter, group of 64 channels, rank tile.  Row r of row tile j of 4 is
// channel (j >> 1) * 32 + (r >> 2) * 8 + (j & 1) * 4 + (r & 3), so that a lane's results are
// 8 neighbouring channels, twice; half j >> 1, row L & 15 of tile j in bytes (j & 1) * 8 on.
constexpr int kAdChain = 128;                  // inputs summed in one go
constexpr int kAdParts = 4, kAdWaves = 4;      // chain c goes to wave c % 16: part, wave of it
inline int64_t ad_rank_tiles(int32_t rank) { return round_up(rank, 16) / 16; }
inline int64_t ad_chains(int32_t K) { return round_up(K, kAdChain) / kAdChain; }
inline int ad_parts(int32_t K) {
    const int64_t c = (ad_chains(K) + kAdWaves - 1) / kAdWaves;
    return (int)(c < kAdParts ? c : kAdParts);
}
inline int64_t ad_a_bytes(int32_t rank, int32_t K) {
    return ad_rank_tiles(rank) * ad_chains(K) * (kAdChain / 32) * 1024;
}
inline int64_t ad_b_bytes(int32_t rank, int32_t N) {
    return round_up(N, 64) / 64 * ad_rank_tiles(rank) * 2048;
}
// What a plan holds, in int32 from its start: records of tiles of up to `tile` tokens
// of one adapter (adapter, place of the first in the order, tokens, 0, then the tokens,
// the last one repeated), no tokens in those past the last; then the sort's own arrays,
// among them the order: tokens by adapter, those without one last.  Tiles of 64, which the
// kernels for many tokens take whole, where a slot has 32 tokens or more.
struct AdPlan {
    int64_t order, ids, counts, offsets, inv, ws, total;
    int64_t tiles;      // records
    int tile, rec;      // tokens and int32 of a record
};
inline AdPlan ad_plan(int64_t T, int32_t n, int tile) {
    AdPlan p;
    p.tile = tile;
    p.rec = 4 + p.tile;
    p.tiles = T / p.tile + (T < n + 1 ? T : n + 1);
    p.order = p.tiles * p.rec;
    p.ids = p.order + round_up(T, 4);
    p.counts = p.ids + round_up(T, 4);
    p.offsets = p.counts + round_up(n + 1, 4);
    p.inv = p.offsets + round_up(n + 2, 4);
    p.ws = p.inv + round_up(T, 4);
    p.total = p.ws + (int64_t)permute_ws_most_bytes(T, 1, n + 1) / 4;
    return p;
}
inline AdPlan ad_plan(int64_t T, int32_t n) {
    return ad_plan(T, n, T >= 1024 && T >= 32 * (int64_t)n ? 64 : 16);
}
int launch_adapter_plan(const int32_t* ids, int64_t T, int32_t n, int32_t* plan, void* stream);
int launch_pack_adapter(const moe_adapters& S, int32_t slot, const void* a, int64_t lda,
                        const void* b, int64_t ldb, int32_t rank, float scale, void* stream);
size_t add_adapters_ws_bytes(const moe_adapters& S, int64_t T);
int launch_add_adapters(const moe_adapters& S, const void* x, int32_t x_dtype, int64_t ldx,
                        const float* x_scale, const int32_t* plan, int64_t T, const void* y,
                        void* out, int32_t y_dtype, int64_t ldy, int64_t ldo, float* h,
                        void* stream);
int launch_probe_read(const void* buf, size_t bytes, uint32_t* sink, int blocks, void* stream);

}  // namespace moeq
