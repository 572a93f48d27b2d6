// Argument checks that the operators' host files share (zero_train_abi.cpp,
// zero_model_abi.cpp): types, sizes, arrays, overlap.
#pragma once

#include <stdint.h>

#include "zero_host.h"
#include "zero_train.h"

namespace zero {
namespace checks {

constexpr int64_t kMaxGrid = 0x7fffffff;   // workgroups of one call, in one launch or several
constexpr int64_t kMaxBytes = int64_t{1} << 56;

// A strided array of one call: what overlap checks and messages need.
struct Array {
    const char* name;
    const void* p;
    int64_t bytes;   // first byte to one behind the last
    int64_t row = 0, stride = 0;  // bytes of a row, and from one to the next
};

inline int64_t elem_size(int32_t dtype) { return dtype == ZERO_F32 ? 4 : 2; }

inline int check_dtype(int32_t dtype, const char* who, const char* name) {
    if (dtype != ZERO_F32 && dtype != ZERO_F16 && dtype != ZERO_BF16)
        return fail(ZERO_EINVAL, "%s: %s = %d is no element type", who, name, dtype);
    return ZERO_OK;
}

inline int check_fmt(int32_t fmt, const char* who, const char* name) {
    if (fmt != ZERO_E4M3 && fmt != ZERO_E5M2)
        return fail(ZERO_EINVAL, "%s: %s = %d is no 8-bit format", who, name, fmt);
    return ZERO_OK;
}

inline int check_size(int64_t n, const char* who, const char* name) {
    if (n < 0) return fail(ZERO_EINVAL, "%s: %s = %lld < 0", who, name, static_cast<long long>(n));
    return ZERO_OK;
}

// rows x cols elements of `size` bytes, rows ld apart; fills out->bytes.
inline int check_array(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size,
                       uintptr_t alignment, const char* who, const char* name, Array* out) {
    *out = Array{name, p, 0, 0, 0};
    if (ld < cols)
        return fail(ZERO_EINVAL, "%s: ld of %s = %lld is less than a row's %lld", who, name,
                    static_cast<long long>(ld), static_cast<long long>(cols));
    int64_t span = 0;
    if (rows > 0 && cols > 0 &&
        (__builtin_mul_overflow(rows - 1, ld, &span) || span > kMaxBytes || cols > kMaxBytes ||
         (span + cols) > kMaxBytes / size))
        return fail(ZERO_EINVAL, "%s: %s is too large", who, name);
    if (rows == 0 || cols == 0) return ZERO_OK;  // nothing is touched
    if (!p) return fail(ZERO_EINVAL, "%s: %s is NULL", who, name);
    if (!aligned(p, alignment))
        return fail(ZERO_EALIGN, "%s: %s is not %d-byte aligned", who, name,
                    static_cast<int>(alignment));
    out->bytes = (span + cols) * size;
    out->row = cols * size;
    if (rows > 1) out->stride = ld * size;  // in range: the rows' span is
    return ZERO_OK;
}

inline int check_elements(const void* p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype,
                          const char* who, const char* name, Array* out) {
    if (int rc = check_dtype(dtype, who, name)) return rc;
    const int64_t size = elem_size(dtype);
    return check_array(p, rows, cols, ld, size, static_cast<uintptr_t>(size), who, name, out);
}

// One q8 matrix: 8-bit data and scale bytes.
inline int check_q8(const void* data, int64_t ld, const uint8_t* scales, int64_t ld_s, int64_t rows,
                    int64_t cols, const char* who, const char* data_name, const char* scale_name,
                    Array* data_out, Array* scale_out) {
    const int64_t blocks = (cols + 127) / 128;
    if (ld % 16)
        return fail(ZERO_EALIGN, "%s: ld of %s is not a multiple of 16", who, data_name);
    if (ld_s % 4)
        return fail(ZERO_EALIGN, "%s: ld of %s is not a multiple of 4", who, scale_name);
    if (int rc = check_array(data, rows, blocks * 128, ld, 1, 16, who, data_name, data_out))
        return rc;
    return check_array(scales, rows, (blocks + 3) / 4 * 4, ld_s, 1, 4, who, scale_name, scale_out);
}

// No output shares a byte with an input or with another output.
inline int check_apart(const Array* outs, int n_outs, const Array* ins, int n_ins,
                       const char* who) {
    for (int o = 0; o < n_outs; ++o) {
        for (int i = 0; i < n_ins; ++i)
            if (overlap(outs[o].p, outs[o].bytes, ins[i].p, ins[i].bytes))
                return fail(ZERO_EINVAL, "%s: %s overlaps %s", who, outs[o].name, ins[i].name);
        for (int p = o + 1; p < n_outs; ++p)
            if (overlap(outs[o].p, outs[o].bytes, outs[p].p, outs[p].bytes))
                return fail(ZERO_EINVAL, "%s: %s overlaps %s", who, outs[o].name, outs[p].name);
    }
    return ZERO_OK;
}

inline int check_ctl(const zero_step_control* d_ctl, const char* who) {
    if (!aligned(d_ctl, 8)) return fail(ZERO_EALIGN, "%s: d_ctl is not 8-byte aligned", who);
    return ZERO_OK;
}

// Output `out` is exactly `in`: same first byte, type and row stride.
inline bool same_array(const void* out, int32_t out_dtype, int64_t ld_out, const void* in,
                       int32_t in_dtype, int64_t ld_in) {
    return out && out == in && out_dtype == in_dtype && ld_out == ld_in;
}

}  // namespace checks
}  // namespace zero
