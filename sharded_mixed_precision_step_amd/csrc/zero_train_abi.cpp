// C-ABI host layer of the training operators: argument validation, launches,
// errors.  Every argument is checked before anything is enqueued.
#include <stdint.h>

#include "zero_host.h"
#include "zero_train_internal.h"

namespace {

using zero::aligned;
using zero::fail;
using zero::finite_f;
using zero::hip_fail;
using zero::ok;
using zero::overlap;

constexpr int64_t kMaxGrid = 0x7fffffff;   // workgroups of one call, in one launch or several
constexpr int64_t kMaxTiles = int64_t{1} << 27;  // a band of eight rows of them fits 32 bits
constexpr int64_t kMaxBytes = int64_t{1} << 56;

// A strided array of one call: what overlap checks and messages need.
struct Array {
    const char* name;
    const void* p;
    int64_t bytes;   // first byte to one behind the last
};

int64_t elem_size(int32_t dtype) { return dtype == ZERO_F32 ? 4 : 2; }

int check_dtype(int32_t dtype, const char* who, const char* name) {
    if (dtype != ZERO_F32 && dtype != ZERO_F16 && dtype != ZERO_BF16)
        return fail(ZERO_EINVAL, "%s: %s = %d is no element type", who, name, dtype);
    return ZERO_OK;
}

int check_fmt(int32_t fmt, const char* who, const char* name) {
    if (fmt != ZERO_E4M3 && fmt != ZERO_E5M2)
        return fail(ZERO_EINVAL, "%s: %s = %d is no 8-bit format", who, name, fmt);
    return ZERO_OK;
}

int check_size(int64_t n, const char* who, const char* name) {
    if (n < 0) return fail(ZERO_EINVAL, "%s: %s = %lld < 0", who, name, static_cast<long long>(n));
    return ZERO_OK;
}

// rows x cols elements of `size` bytes, rows ld apart; fills out->bytes.
int check_array(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size,
                uintptr_t alignment, const char* who, const char* name, Array* out) {
    *out = Array{name, p, 0};
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
    return ZERO_OK;
}

int check_elements(const void* p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype,
                   const char* who, const char* name, Array* out) {
    if (int rc = check_dtype(dtype, who, name)) return rc;
    const int64_t size = elem_size(dtype);
    return check_array(p, rows, cols, ld, size, static_cast<uintptr_t>(size), who, name, out);
}

// One q8 matrix: 8-bit data and scale bytes.
int check_q8(const void* data, int64_t ld, const uint8_t* scales, int64_t ld_s, int64_t rows,
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
int check_apart(const Array* outs, int n_outs, const Array* ins, int n_ins, const char* who) {
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

int quantize(const void* const* srcs, int n_srcs, int32_t dtype, int64_t rows, int64_t cols,
             int64_t ld_src, int32_t fmt, void* q, int64_t ld_q, uint8_t* s, int64_t ld_s,
             void* qt, int64_t ld_qt, uint8_t* st, int64_t ld_st, const zero_step_control* ctl,
             hipStream_t stream, const char* who) {
    int rc;
    if ((rc = check_dtype(dtype, who, "dtype")) || (rc = check_fmt(fmt, who, "fmt")) ||
        (rc = check_size(rows, who, "rows")) || (rc = check_size(cols, who, "cols")))
        return rc;
    if (!q != !s) return fail(ZERO_EINVAL, "%s: q and s go together", who);
    if (!qt != !st) return fail(ZERO_EINVAL, "%s: qt and st go together", who);
    if (rows == 0 || cols == 0) return ok();
    if (!q && !qt) return fail(ZERO_EINVAL, "%s: no output is given", who);
    Array in[2], out[4];
    int n_out = 0;
    for (int k = 0; k < n_srcs; ++k)
        if ((rc = check_elements(srcs[k], rows, cols, ld_src, dtype, who, "src", &in[k])))
            return rc;
    if (q) {
        if ((rc = check_q8(q, ld_q, s, ld_s, rows, cols, who, "q", "s", &out[0], &out[1])))
            return rc;
        n_out = 2;
    }
    if (qt) {
        if ((rc = check_q8(qt, ld_qt, st, ld_st, cols, rows, who, "qt", "st", &out[n_out],
                           &out[n_out + 1])))
            return rc;
        n_out += 2;
    }
    if ((rc = check_apart(out, n_out, in, n_srcs, who))) return rc;
    if (zero::quantize_blocks(rows, cols) > kMaxGrid)
        return fail(ZERO_EINVAL, "%s: the matrix is larger than a call's launches cover", who);
    zero::QuantizeArgs a = {};
    a.src[0] = srcs[0];
    a.src[1] = n_srcs > 1 ? srcs[1] : nullptr;
    a.ctl = ctl;
    a.rows = rows; a.cols = cols; a.ld_src = ld_src;
    a.q = static_cast<uint8_t*>(q); a.s = s;
    a.qt = static_cast<uint8_t*>(qt); a.st = st;
    a.ld_q = ld_q; a.ld_s = ld_s; a.ld_qt = ld_qt; a.ld_st = ld_st;
    a.dtype = dtype; a.fmt = fmt;
    const hipError_t e = zero::launch_q8_quantize(a, stream);
    return e == hipSuccess ? ok() : hip_fail(e, who);
}

int check_ctl(const zero_step_control* d_ctl, const char* who) {
    if (!aligned(d_ctl, 8)) return fail(ZERO_EALIGN, "%s: d_ctl is not 8-byte aligned", who);
    return ZERO_OK;
}

int distill(const zero_distill_inputs* in, zero::DistillMode mode, float loss_scale,
            const zero_step_control* ctl, float* loss, float* lse, const float* lse_in, void* grad,
            int64_t ld_grad, hipStream_t stream, const char* who) {
    int rc;
    if (!in) return fail(ZERO_EINVAL, "%s: in is NULL", who);
    if ((rc = check_dtype(in->logits_dtype, who, "logits_dtype")) ||
        (rc = check_dtype(in->top_dtype, who, "top_dtype")) ||
        (rc = check_size(in->rows, who, "rows")))
        return rc;
    if (in->vocab < 1 || in->vocab > 0x7fffffff)
        return fail(ZERO_EINVAL, "%s: vocab = %lld outside [1, 2^31 - 1]", who,
                    static_cast<long long>(in->vocab));
    if (in->index_bytes != 4 && in->index_bytes != 8)
        return fail(ZERO_EINVAL, "%s: index_bytes = %d is neither 4 nor 8", who, in->index_bytes);
    if (in->top < 1) return fail(ZERO_EINVAL, "%s: top = %d < 1", who, in->top);
    if (in->top > ZERO_DISTILL_MAX_TOP)
        return fail(ZERO_ERANGE, "%s: top = %d is above %d", who, in->top, ZERO_DISTILL_MAX_TOP);
    if (!finite_f(in->temperature) || !(in->temperature > 0.0f) ||
        !finite_f(1.442695041f / in->temperature) ||
        !finite_f(in->temperature * in->temperature))
        return fail(ZERO_EINVAL, "%s: temperature = %g is not finite and > 0, or its square or "
                    "log2(e) by it is not finite", who, static_cast<double>(in->temperature));
    if (mode != zero::kDistillForward) {
        if (ctl) {
            if ((rc = check_ctl(ctl, who))) return rc;
        } else if (!finite_f(loss_scale) || !(loss_scale > 0.0f)) {
            return fail(ZERO_EINVAL, "%s: loss_scale = %g is not finite and > 0", who,
                        static_cast<double>(loss_scale));
        }
    } else if (!loss && !lse) {
        return fail(ZERO_EINVAL, "%s: no output is given", who);
    }
    if (in->rows == 0) return ok();
    Array ins[5], outs[3];
    int n_in = 3, n_out = 0;
    if ((rc = check_elements(in->logits, in->rows, in->vocab, in->ld_logits, in->logits_dtype, who,
                             "logits", &ins[0])) ||
        (rc = check_array(in->top_index, in->rows, in->top, in->ld_top, in->index_bytes,
                          static_cast<uintptr_t>(in->index_bytes), who, "top_index", &ins[1])) ||
        (rc = check_elements(in->top_logit, in->rows, in->top, in->ld_top, in->top_dtype, who,
                             "top_logit", &ins[2])))
        return rc;
    if (in->row_weight &&
        (rc = check_array(in->row_weight, 1, in->rows, in->rows, 4, 4, who, "row_weight",
                          &ins[n_in++])))
        return rc;
    if (mode == zero::kDistillBackward &&
        (rc = check_array(lse_in, 1, in->rows, in->rows, 4, 4, who, "lse", &ins[n_in++])))
        return rc;
    if (loss &&
        (rc = check_array(loss, 1, in->rows, in->rows, 4, 4, who, "loss", &outs[n_out++])))
        return rc;
    if (lse && (rc = check_array(lse, 1, in->rows, in->rows, 4, 4, who, "lse", &outs[n_out++])))
        return rc;
    if (mode != zero::kDistillForward) {
        Array g;
        if ((rc = check_elements(grad, in->rows, in->vocab, ld_grad, in->logits_dtype, who, "grad",
                                 &g)))
            return rc;
        const bool in_place = grad == in->logits;
        if (in_place && ld_grad != in->ld_logits)
            return fail(ZERO_EINVAL, "%s: grad is the logits, with another row stride", who);
        if ((rc = check_apart(&g, 1, ins + (in_place ? 1 : 0), n_in - (in_place ? 1 : 0), who)) ||
            (rc = check_apart(outs, n_out, &g, 1, who)))
            return rc;
    }
    if ((rc = check_apart(outs, n_out, ins, n_in, who))) return rc;
    if (in->rows > kMaxGrid)
        return fail(ZERO_EINVAL, "%s: more rows than a call's launches cover", who);
    zero::DistillArgs a = {};
    a.logits = in->logits; a.index = in->top_index; a.top_logit = in->top_logit;
    a.weight = in->row_weight;
    a.rows = in->rows; a.vocab = in->vocab; a.ld = in->ld_logits; a.ld_top = in->ld_top;
    a.dtype = in->logits_dtype; a.top_dtype = in->top_dtype; a.index_bytes = in->index_bytes;
    a.top = in->top;
    a.tau = in->temperature;
    a.S = loss_scale;
    a.ctl = ctl;
    a.loss = loss; a.lse = lse; a.lse_in = lse_in;
    a.grad = grad; a.ld_grad = ld_grad;
    const hipError_t e = zero::launch_distill(a, mode, stream);
    return e == hipSuccess ? ok() : hip_fail(e, who);
}

int check_norm_cols(int64_t cols, const char* who) {
    if (cols < 1) return fail(ZERO_EINVAL, "%s: cols = %lld < 1", who, static_cast<long long>(cols));
    if (cols > ZERO_NORM_MAX_COLS)
        return fail(ZERO_ERANGE, "%s: cols = %lld is above %d", who, static_cast<long long>(cols),
                    ZERO_NORM_MAX_COLS);
    return ZERO_OK;
}

// Output `out` is exactly `in`: same first byte, type and row stride.
bool same_array(const void* out, int32_t out_dtype, int64_t ld_out, const void* in,
                int32_t in_dtype, int64_t ld_in) {
    return out && out == in && out_dtype == in_dtype && ld_out == ld_in;
}

}  // namespace

extern "C" {

int zero_q8_quantize(const void* src, int32_t dtype, int64_t rows, int64_t cols, int64_t ld_src,
                     int32_t fmt, void* q, int64_t ld_q, uint8_t* s, int64_t ld_s, void* qt,
                     int64_t ld_qt, uint8_t* st, int64_t ld_st, void* stream) {
    return quantize(&src, 1, dtype, rows, cols, ld_src, fmt, q, ld_q, s, ld_s, qt, ld_qt, st, ld_st,
                    nullptr, static_cast<hipStream_t>(stream), "zero_q8_quantize");
}

int zero_q8_quantize_ctl(const void* const* srcs_fp16, int64_t rows, int64_t cols, int64_t ld_src,
                         int32_t fmt, void* q, int64_t ld_q, uint8_t* s, int64_t ld_s, void* qt,
                         int64_t ld_qt, uint8_t* st, int64_t ld_st,
                         const zero_step_control* d_ctl, void* stream) {
    const char* who = "zero_q8_quantize_ctl";
    if (!srcs_fp16) return fail(ZERO_EINVAL, "%s: srcs_fp16 is NULL", who);
    if (!d_ctl) return fail(ZERO_EINVAL, "%s: d_ctl is NULL", who);
    if (int rc = check_ctl(d_ctl, who)) return rc;
    return quantize(srcs_fp16, 2, ZERO_F16, rows, cols, ld_src, fmt, q, ld_q, s, ld_s, qt, ld_qt,
                    st, ld_st, d_ctl, static_cast<hipStream_t>(stream), who);
}

int zero_q8_gemm(const void* a, int32_t fmt_a, int64_t ld_a, const uint8_t* sa, int64_t ld_sa,
                 const void* b, int32_t fmt_b, int64_t ld_b, const uint8_t* sb, int64_t ld_sb,
                 int64_t m, int64_t n, int64_t k, void* c, int32_t c_dtype, int64_t ld_c,
                 int32_t accumulate, void* stream) {
    const char* who = "zero_q8_gemm";
    int rc;
    if ((rc = check_fmt(fmt_a, who, "fmt_a")) || (rc = check_fmt(fmt_b, who, "fmt_b")) ||
        (rc = check_dtype(c_dtype, who, "c_dtype")) || (rc = check_size(m, who, "m")) ||
        (rc = check_size(n, who, "n")) || (rc = check_size(k, who, "k")))
        return rc;
    if (accumulate != 0 && accumulate != 1)
        return fail(ZERO_EINVAL, "%s: accumulate = %d is neither 0 nor 1", who, accumulate);
    if (m == 0 || n == 0) return ok();
    if (k == 0) {  // nothing of a and b is there
        a = b = nullptr;
        sa = sb = nullptr;
        ld_a = ld_b = ld_sa = ld_sb = 0;
    }
    if (k > ZERO_Q8_MAX_LD || ld_a > ZERO_Q8_MAX_LD || ld_b > ZERO_Q8_MAX_LD ||
        ld_sa > ZERO_Q8_MAX_LD || ld_sb > ZERO_Q8_MAX_LD)
        return fail(ZERO_ERANGE, "%s: k or a row stride is above %d", who, ZERO_Q8_MAX_LD);
    Array ins[4], out;
    if ((rc = check_q8(a, ld_a, sa, ld_sa, m, k, who, "a", "sa", &ins[0], &ins[1])) ||
        (rc = check_q8(b, ld_b, sb, ld_sb, n, k, who, "b", "sb", &ins[2], &ins[3])) ||
        (rc = check_elements(c, m, n, ld_c, c_dtype, who, "c", &out)) ||
        (rc = check_apart(&out, 1, ins, 4, who)))
        return rc;
    zero::GemmArgs g = {};
    g.a = static_cast<const uint8_t*>(a); g.sa = sa;
    g.b = static_cast<const uint8_t*>(b); g.sb = sb;
    g.ld_a = ld_a; g.ld_sa = ld_sa; g.ld_b = ld_b; g.ld_sb = ld_sb;
    g.m = m; g.n = n;
    g.kblocks = static_cast<int32_t>((k + 127) / 128);
    g.fmt_a = fmt_a; g.fmt_b = fmt_b; g.c_dtype = c_dtype; g.accumulate = accumulate;
    g.c = c; g.ld_c = ld_c;
    if (zero::gemm_tiles(m, n) > kMaxTiles)
        return fail(ZERO_EINVAL, "%s: c is larger than a call's launches cover", who);
    const hipError_t e = zero::launch_q8_gemm(g, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, who);
}

int zero_rmsnorm(const void* x, int32_t x_dtype, int64_t ld_x, const void* residual,
                 int32_t r_dtype, int64_t ld_r, const void* weight, int32_t w_dtype, int64_t rows,
                 int64_t cols, float eps, void* h, int64_t ld_h, void* y, int32_t y_dtype,
                 int64_t ld_y, void* q, int32_t fmt, int64_t ld_q, uint8_t* s, int64_t ld_s,
                 float* rstd, void* stream) {
    const char* who = "zero_rmsnorm";
    int rc;
    if ((rc = check_size(rows, who, "rows")) || (rc = check_norm_cols(cols, who))) return rc;
    if (!finite_f(eps) || eps < 0.0f)
        return fail(ZERO_EINVAL, "%s: eps = %g is not finite and >= 0", who,
                    static_cast<double>(eps));
    if (!q != !s) return fail(ZERO_EINVAL, "%s: q and s go together", who);
    if (q && (rc = check_fmt(fmt, who, "fmt"))) return rc;
    if (h && !residual) return fail(ZERO_EINVAL, "%s: h is given without a residual", who);
    Array ins[3], outs[5];
    int n_in = 0, n_out = 0;
    const int64_t live = rows > 0 ? 1 : 0;
    if ((rc = check_elements(x, rows, cols, ld_x, x_dtype, who, "x", &ins[n_in++])) ||
        (rc = check_elements(weight, live, cols, cols, w_dtype, who, "weight", &ins[n_in++])))
        return rc;
    if (residual &&
        (rc = check_elements(residual, rows, cols, ld_r, r_dtype, who, "residual", &ins[n_in++])))
        return rc;
    if (rows == 0) return ok();
    if (!h && !y && !q && !rstd) return fail(ZERO_EINVAL, "%s: no output is given", who);
    bool h_is_x = false, h_is_r = false, y_is_x = false;
    if (h) {
        if ((rc = check_elements(h, rows, cols, ld_h, r_dtype, who, "h", &outs[n_out++])))
            return rc;
        h_is_x = same_array(h, r_dtype, ld_h, x, x_dtype, ld_x);
        h_is_r = same_array(h, r_dtype, ld_h, residual, r_dtype, ld_r);
    }
    if (y) {
        if ((rc = check_elements(y, rows, cols, ld_y, y_dtype, who, "y", &outs[n_out++])))
            return rc;
        y_is_x = same_array(y, y_dtype, ld_y, x, x_dtype, ld_x);
    }
    if (q) {
        if ((rc = check_q8(q, ld_q, s, ld_s, rows, cols, who, "q", "s", &outs[n_out],
                           &outs[n_out + 1])))
            return rc;
        n_out += 2;
    }
    if (rstd &&
        (rc = check_array(rstd, 1, rows, rows, 4, 4, who, "rstd", &outs[n_out++])))
        return rc;
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i) {
            const bool is_h = h && o == 0, is_y = y && o == (h ? 1 : 0);
            if (is_h && ((i == 0 && h_is_x) || (i == 2 && h_is_r))) continue;
            if (is_y && i == 0 && y_is_x) continue;
            if ((rc = check_apart(&outs[o], 1, &ins[i], 1, who))) return rc;
        }
    }
    if ((rc = check_apart(outs, n_out, nullptr, 0, who))) return rc;
    if (rows > kMaxGrid) return fail(ZERO_EINVAL, "%s: more rows than a call's launches cover", who);
    zero::NormArgs a = {};
    a.x = x; a.res = residual; a.weight = weight;
    a.ld_x = ld_x; a.ld_r = ld_r; a.ld_h = ld_h; a.ld_y = ld_y; a.ld_q = ld_q; a.ld_s = ld_s;
    a.rows = rows;
    a.cols = static_cast<int32_t>(cols);
    a.x_dtype = x_dtype; a.r_dtype = r_dtype; a.w_dtype = w_dtype; a.y_dtype = y_dtype;
    a.fmt = fmt;
    a.eps = eps;
    a.h = h; a.y = y; a.q = static_cast<uint8_t*>(q); a.s = s; a.rstd = rstd;
    const hipError_t e = zero::launch_rmsnorm(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, who);
}

int64_t zero_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
    const char* who = "zero_rmsnorm_backward_workspace";
    if (check_size(rows, who, "rows") || check_norm_cols(cols, who)) return -1;
    ok();
    return 4 * cols * zero::norm_backward_parts(rows, static_cast<int32_t>(cols));
}

int zero_rmsnorm_backward(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* h,
                          int32_t h_dtype, int64_t ld_h, const void* weight, int32_t w_dtype,
                          const float* rstd, const void* dresidual, int32_t dr_dtype,
                          int64_t ld_dr, int64_t rows, int64_t cols, void* dx, int32_t dx_dtype,
                          int64_t ld_dx, void* dw, int32_t dw_dtype, void* workspace,
                          int64_t workspace_bytes, void* stream) {
    const char* who = "zero_rmsnorm_backward";
    int rc;
    if ((rc = check_size(rows, who, "rows")) || (rc = check_norm_cols(cols, who))) return rc;
    const int64_t live = rows > 0 ? 1 : 0;
    Array ins[5], outs[3];
    int n_in = 4, n_out = 1;
    if ((rc = check_elements(dy, rows, cols, ld_dy, dy_dtype, who, "dy", &ins[0])) ||
        (rc = check_elements(h, rows, cols, ld_h, h_dtype, who, "h", &ins[1])) ||
        (rc = check_elements(weight, live, cols, cols, w_dtype, who, "weight", &ins[2])) ||
        (rc = check_array(rstd, live, rows, rows, 4, 4, who, "rstd", &ins[3])) ||
        (rc = check_elements(dx, rows, cols, ld_dx, dx_dtype, who, "dx", &outs[0])))
        return rc;
    if (dresidual && (rc = check_elements(dresidual, rows, cols, ld_dr, dr_dtype, who, "dresidual",
                                          &ins[n_in++])))
        return rc;
    const int64_t parts = zero::norm_backward_parts(rows, static_cast<int32_t>(cols));
    if (dw) {
        if ((rc = check_elements(dw, 1, cols, cols, dw_dtype, who, "dw", &outs[n_out++])))
            return rc;
        if (workspace_bytes < 4 * cols * parts)
            return fail(ZERO_ERANGE, "%s: workspace_bytes = %lld, %lld are needed", who,
                        static_cast<long long>(workspace_bytes),
                        static_cast<long long>(4 * cols * parts));
        if ((rc = check_array(workspace, parts, cols, cols, 4, 16, who, "workspace",
                              &outs[n_out++])))
            return rc;
    }
    const bool is_dy = same_array(dx, dx_dtype, ld_dx, dy, dy_dtype, ld_dy);
    const bool is_h = same_array(dx, dx_dtype, ld_dx, h, h_dtype, ld_h);
    const bool is_dr = dresidual && same_array(dx, dx_dtype, ld_dx, dresidual, dr_dtype, ld_dr);
    for (int o = 0; o < n_out; ++o)
        for (int i = 0; i < n_in; ++i) {
            if (o == 0 && ((i == 0 && is_dy) || (i == 1 && is_h) || (i == 4 && is_dr))) continue;
            if ((rc = check_apart(&outs[o], 1, &ins[i], 1, who))) return rc;
        }
    if ((rc = check_apart(outs, n_out, nullptr, 0, who))) return rc;
    zero::NormBackwardArgs a = {};
    a.dy = dy; a.h = h; a.weight = weight; a.dres = dresidual; a.rstd = rstd;
    a.ld_dy = ld_dy; a.ld_h = ld_h; a.ld_dr = ld_dr; a.ld_dx = ld_dx;
    a.rows = rows;
    a.cols = static_cast<int32_t>(cols);
    a.dy_dtype = dy_dtype; a.h_dtype = h_dtype; a.w_dtype = w_dtype; a.dr_dtype = dr_dtype;
    a.dx_dtype = dx_dtype; a.dw_dtype = dw_dtype;
    a.dx = dx; a.dw = dw;
    a.parts = dw ? static_cast<float*>(workspace) : nullptr;
    const hipError_t e = zero::launch_rmsnorm_backward(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, who);
}

int zero_distill_forward(const zero_distill_inputs* in, float* loss, float* lse, void* stream) {
    return distill(in, zero::kDistillForward, 1.0f, nullptr, loss, lse, nullptr, nullptr, 0,
                   static_cast<hipStream_t>(stream), "zero_distill_forward");
}

int zero_distill_backward(const zero_distill_inputs* in, const float* lse, float loss_scale,
                          const zero_step_control* d_ctl, void* grad, int64_t ld_grad,
                          void* stream) {
    return distill(in, zero::kDistillBackward, loss_scale, d_ctl, nullptr, nullptr, lse, grad,
                   ld_grad, static_cast<hipStream_t>(stream), "zero_distill_backward");
}

int zero_distill(const zero_distill_inputs* in, float loss_scale, const zero_step_control* d_ctl,
                 float* loss, float* lse, void* grad, int64_t ld_grad, void* stream) {
    return distill(in, zero::kDistillBoth, loss_scale, d_ctl, loss, lse, nullptr, grad, ld_grad,
                   static_cast<hipStream_t>(stream), "zero_distill");
}

}  // extern "C"
