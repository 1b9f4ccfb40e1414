// Checks that the C entries of operands of several element types share.
#pragma once

#include <cstdint>
#include <string>

#include "internal.h"

namespace moeq {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRows = (int64_t)1 << 31;   // grid rows of one launch
constexpr int32_t kMaxDim = 1 << 24;             // widths

inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline bool float_dt(int dt) { return dt == MOE_DT_F32 || dt == MOE_DT_BF16 || dt == MOE_DT_F16; }
inline int64_t dt_bytes(int dt) { return dt == MOE_DT_F32 ? 4 : dt == MOE_DT_I8 ? 1 : 2; }

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline int bad(const std::string& fn, const char* what) { return fail(MOE_EINVAL, fn + ": " + what); }

// Operand rows of H elements: the type, the pointer's natural alignment and
// the row stride; vec8 is cleared if a row may start off a 16-byte border.
inline int check_rows(const std::string& fn, const char* name, const void* p, int dt, int64_t ld,
               int64_t H, bool& vec8) {
    if (!float_dt(dt))
        return fail(MOE_EUNSUPPORTED, fn + ": " + name + " has an unknown element type");
    if (!aligned(p, (uintptr_t)dt_bytes(dt)))
        return fail(MOE_EINVAL, fn + ": " + name + " is not aligned to its element type");
    if (ld < H) return fail(MOE_EINVAL, fn + ": the row stride of " + name + " is below the width");
    vec8 = vec8 && aligned(p, 16) && ld * dt_bytes(dt) % 16 == 0;
    return MOE_OK;
}

inline int check_codes(const std::string& fn, const char* name, const void* q, int64_t ldq, int64_t K) {
    if (!aligned(q, 16) || ldq % 16 || ldq < round_up(K, kI8TileK))
        return fail(MOE_EINVAL, fn + ": " + name +
                                    " needs 16-byte aligned rows of at least the width rounded up "
                                    "to 64 codes");
    return MOE_OK;
}

}  // namespace moeq
