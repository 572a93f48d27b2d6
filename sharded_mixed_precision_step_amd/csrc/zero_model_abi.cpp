// C-ABI host layer of zero_model.h's operators: argument validation, launches,
// errors.  Every argument is checked before anything is enqueued.
#include <stdint.h>

#include "zero_model_internal.h"
#include "zero_train_checks.h"

namespace {

using namespace zero::checks;
using zero::fail;
using zero::finite_f;
using zero::hip_fail;
using zero::ok;

// Two arrays of one row stride that are different column ranges of one matrix.
bool side_by_side(const Array& a, const Array& b) {
    if (a.stride <= 0 || a.stride != b.stride) return false;
    const uintptr_t stride = static_cast<uintptr_t>(a.stride);
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p) % stride;
    const uintptr_t y = reinterpret_cast<uintptr_t>(b.p) % stride;
    const int64_t d = static_cast<int64_t>((y + stride - x) % stride);
    return d >= a.row && a.stride - d >= b.row;
}

int check_two(const Array& out, const Array& other, const char* who) {
    return side_by_side(out, other) ? ZERO_OK : check_apart(&out, 1, &other, 1, who);
}

// No output shares a byte with an input, inputs i with bit i of `same` excepted.
int check_apart_but(const Array& out, const Array* ins, int n_ins, uint32_t same, const char* who) {
    for (int i = 0; i < n_ins; ++i) {
        if (same >> i & 1) continue;
        if (int rc = check_two(out, ins[i], who)) return rc;
    }
    return ZERO_OK;
}

// No two outputs share a byte.
int check_outputs(const Array* outs, int n_outs, const char* who) {
    for (int o = 0; o < n_outs; ++o)
        for (int p = o + 1; p < n_outs; ++p)
            if (int rc = check_two(outs[o], outs[p], who)) return rc;
    return ZERO_OK;
}

int check_ids(const void* ids, int32_t id_bytes, int64_t n, const char* who, Array* out) {
    if (id_bytes != 4 && id_bytes != 8)
        return fail(ZERO_EINVAL, "%s: id_bytes = %d is neither 4 nor 8", who, id_bytes);
    return check_array(ids, 1, n, n, id_bytes, static_cast<uintptr_t>(id_bytes), who, "ids", out);
}

int check_positive(int64_t n, const char* who, const char* name) {
    if (n < 1 || n > 0x7fffffff)
        return fail(ZERO_EINVAL, "%s: %s = %lld outside [1, 2^31 - 1]", who, name,
                    static_cast<long long>(n));
    return ZERO_OK;
}

int check_vector(const void* p, int64_t n, const char* who, const char* name, Array* out) {
    return check_array(p, 1, n, n, 4, 4, who, name, out);
}

int too_many(const char* who) {
    return fail(ZERO_EINVAL, "%s: more rows than a call's launches cover", who);
}

int embed(const void* const* tables, int n_tables, int32_t t_dtype, int64_t vocab, int64_t cols,
          int64_t ld_t, const void* ids, int32_t id_bytes, int64_t tokens, float scale, void* y,
          int32_t y_dtype, int64_t ld_y, const zero_step_control* ctl, hipStream_t stream,
          const char* who) {
    int rc;
    if ((rc = check_dtype(t_dtype, who, "t_dtype")) || (rc = check_dtype(y_dtype, who, "y_dtype")) ||
        (rc = check_size(tokens, who, "tokens")) || (rc = check_positive(vocab, who, "vocab")) ||
        (rc = check_positive(cols, who, "cols")))
        return rc;
    if (!finite_f(scale))
        return fail(ZERO_EINVAL, "%s: scale = %g is not finite", who, static_cast<double>(scale));
    if (id_bytes != 4 && id_bytes != 8)
        return fail(ZERO_EINVAL, "%s: id_bytes = %d is neither 4 nor 8", who, id_bytes);
    if (tokens == 0) return ok();
    Array ins[3], out;
    int n_in = 0;
    if ((rc = check_ids(ids, id_bytes, tokens, who, &ins[n_in++]))) return rc;
    for (int k = 0; k < n_tables; ++k)
        if ((rc = check_elements(tables[k], vocab, cols, ld_t, t_dtype, who, "table",
                                 &ins[n_in++])))
            return rc;
    if ((rc = check_elements(y, tokens, cols, ld_y, y_dtype, who, "y", &out)) ||
        (rc = check_apart_but(out, ins, n_in, 0u, who)))
        return rc;
    if (tokens > kMaxGrid || zero::embed_blocks(tokens, cols) > kMaxGrid) return too_many(who);
    zero::EmbedArgs a = {};
    a.table[0] = tables[0];
    a.table[1] = n_tables > 1 ? tables[1] : nullptr;
    a.ctl = ctl;
    a.ids = ids; a.id_bytes = id_bytes;
    a.tokens = tokens; a.vocab = vocab; a.cols = cols; a.ld_t = ld_t; a.ld_y = ld_y;
    a.t_dtype = t_dtype; a.y_dtype = y_dtype;
    a.scale = scale;
    a.y = y;
    const hipError_t e = zero::launch_embed(a, stream);
    return e == hipSuccess ? ok() : hip_fail(e, who);
}

int check_embed_backward_sizes(int64_t tokens, int64_t vocab, int64_t cols, const char* who) {
    int rc;
    if ((rc = check_size(tokens, who, "tokens")) || (rc = check_positive(vocab, who, "vocab")) ||
        (rc = check_positive(cols, who, "cols")))
        return rc;
    if (tokens > ZERO_EMBED_MAX_TOKENS)
        return fail(ZERO_ERANGE, "%s: tokens = %lld is above %d", who,
                    static_cast<long long>(tokens), ZERO_EMBED_MAX_TOKENS);
    return ZERO_OK;
}

int check_layernorm_cols(int64_t cols, const char* who) {
    if (cols < 1) return fail(ZERO_EINVAL, "%s: cols = %lld < 1", who, static_cast<long long>(cols));
    if (cols > ZERO_LAYERNORM_MAX_COLS)
        return fail(ZERO_ERANGE, "%s: cols = %lld is above %d", who, static_cast<long long>(cols),
                    ZERO_LAYERNORM_MAX_COLS);
    return ZERO_OK;
}

int check_kind(int32_t kind, const char* who) {
    if (kind != ZERO_SILU && kind != ZERO_GELU && kind != ZERO_GELU_TANH)
        return fail(ZERO_EINVAL, "%s: kind = %d is no activation", who, kind);
    return ZERO_OK;
}

// What both log probability calls ask of the logits, the ids and the
// temperature; rows > 0.
int check_logits(const void* logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab,
                 const void* ids, int32_t id_bytes, const char* who, Array* ins, int* n_in) {
    int rc;
    if ((rc = check_elements(logits, rows, vocab, ld, dtype, who, "logits", &ins[(*n_in)++])))
        return rc;
    if (ids && (rc = check_ids(ids, id_bytes, rows, who, &ins[(*n_in)++]))) return rc;
    return ZERO_OK;
}

int check_logprob_values(int32_t dtype, int64_t rows, int64_t vocab, const void* ids,
                         int32_t id_bytes, float temperature, const char* who) {
    int rc;
    if ((rc = check_dtype(dtype, who, "dtype")) || (rc = check_size(rows, who, "rows")) ||
        (rc = check_positive(vocab, who, "vocab")))
        return rc;
    if (ids && id_bytes != 4 && id_bytes != 8)
        return fail(ZERO_EINVAL, "%s: id_bytes = %d is neither 4 nor 8", who, id_bytes);
    if (!finite_f(temperature) || !(temperature > 0.0f) || !finite_f(1.442695041f / temperature))
        return fail(ZERO_EINVAL, "%s: temperature = %g is not finite and > 0, or log2(e) by it is "
                    "not finite", who, static_cast<double>(temperature));
    return ZERO_OK;
}

}  // namespace

extern "C" {

int zero_embed(const void* table, int32_t t_dtype, int64_t vocab, int64_t cols, int64_t ld_t,
               const void* ids, int32_t id_bytes, int64_t tokens, float scale, void* y,
               int32_t y_dtype, int64_t ld_y, void* stream) {
    return embed(&table, 1, t_dtype, vocab, cols, ld_t, ids, id_bytes, tokens, scale, y, y_dtype,
                 ld_y, nullptr, static_cast<hipStream_t>(stream), "zero_embed");
}

int zero_embed_ctl(const void* const* tables_fp16, int64_t vocab, int64_t cols, int64_t ld_t,
                   const void* ids, int32_t id_bytes, int64_t tokens, float scale, void* y,
                   int32_t y_dtype, int64_t ld_y, const zero_step_control* d_ctl, void* stream) {
    const char* who = "zero_embed_ctl";
    if (!tables_fp16) return fail(ZERO_EINVAL, "%s: tables_fp16 is NULL", who);
    if (!d_ctl) return fail(ZERO_EINVAL, "%s: d_ctl is NULL", who);
    if (int rc = check_ctl(d_ctl, who)) return rc;
    return embed(tables_fp16, 2, ZERO_F16, vocab, cols, ld_t, ids, id_bytes, tokens, scale, y,
                 y_dtype, ld_y, d_ctl, static_cast<hipStream_t>(stream), who);
}

int64_t zero_embed_backward_workspace(int64_t tokens, int64_t vocab, int64_t cols) {
    if (check_embed_backward_sizes(tokens, vocab, cols, "zero_embed_backward_workspace")) return -1;
    ok();
    return zero::embed_workspace(tokens, cols).bytes;
}

int zero_embed_backward(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* ids,
                        int32_t id_bytes, int64_t tokens, int64_t vocab, int64_t cols, float scale,
                        void* dtable, int32_t dt_dtype, int64_t ld_dt, int32_t accumulate,
                        void* workspace, int64_t workspace_bytes, void* stream) {
    const char* who = "zero_embed_backward";
    int rc;
    if ((rc = check_dtype(dy_dtype, who, "dy_dtype")) ||
        (rc = check_dtype(dt_dtype, who, "dt_dtype")) ||
        (rc = check_embed_backward_sizes(tokens, vocab, cols, who)))
        return rc;
    if (id_bytes != 4 && id_bytes != 8)
        return fail(ZERO_EINVAL, "%s: id_bytes = %d is neither 4 nor 8", who, id_bytes);
    if (!finite_f(scale))
        return fail(ZERO_EINVAL, "%s: scale = %g is not finite", who, static_cast<double>(scale));
    if (accumulate != 0 && accumulate != 1)
        return fail(ZERO_EINVAL, "%s: accumulate = %d is neither 0 nor 1", who, accumulate);
    Array ins[2], outs[2];
    int n_in = 0, n_out = 0;
    if ((rc = check_elements(dtable, vocab, cols, ld_dt, dt_dtype, who, "dtable", &outs[n_out++])))
        return rc;
    if (tokens > 0) {
        if ((rc = check_elements(dy, tokens, cols, ld_dy, dy_dtype, who, "dy", &ins[n_in++])) ||
            (rc = check_ids(ids, id_bytes, tokens, who, &ins[n_in++])))
            return rc;
        const int64_t need = zero::embed_workspace(tokens, cols).bytes;
        if (workspace_bytes < need)
            return fail(ZERO_ERANGE, "%s: workspace_bytes = %lld, %lld are needed", who,
                        static_cast<long long>(workspace_bytes), static_cast<long long>(need));
        if ((rc = check_array(workspace, 1, need, need, 1, 16, who, "workspace", &outs[n_out++])))
            return rc;
    }
    for (int o = 0; o < n_out; ++o)
        if ((rc = check_apart_but(outs[o], ins, n_in, 0u, who))) return rc;
    if ((rc = check_outputs(outs, n_out, who))) return rc;
    if (zero::embed_backward_blocks(tokens, vocab, cols, ld_dt, dt_dtype) > kMaxGrid)
        return too_many(who);
    zero::EmbedBackwardArgs a = {};
    a.dy = dy; a.ids = ids;
    a.tokens = tokens; a.vocab = vocab; a.cols = cols; a.ld_dy = ld_dy; a.ld_dt = ld_dt;
    a.id_bytes = id_bytes; a.dy_dtype = dy_dtype; a.dt_dtype = dt_dtype; a.accumulate = accumulate;
    a.scale = scale;
    a.dtable = dtable;
    a.workspace = static_cast<char*>(workspace);
    const hipError_t e = zero::launch_embed_backward(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, who);
}

int zero_layernorm(const void* x, int32_t x_dtype, int64_t ld_x, const void* residual,
                   int32_t r_dtype, int64_t ld_r, const void* weight, const void* bias,
                   int32_t w_dtype, int64_t rows, int64_t cols, float eps, void* h, int64_t ld_h,
                   void* y, int32_t y_dtype, int64_t ld_y, void* q, int32_t fmt, int64_t ld_q,
                   uint8_t* s, int64_t ld_s, float* mean, float* rstd, void* stream) {
    const char* who = "zero_layernorm";
    int rc;
    if ((rc = check_size(rows, who, "rows")) || (rc = check_layernorm_cols(cols, who))) return rc;
    if (!finite_f(eps) || eps < 0.0f)
        return fail(ZERO_EINVAL, "%s: eps = %g is not finite and >= 0", who,
                    static_cast<double>(eps));
    if (!q != !s) return fail(ZERO_EINVAL, "%s: q and s go together", who);
    if (q && (rc = check_fmt(fmt, who, "fmt"))) return rc;
    if (h && !residual) return fail(ZERO_EINVAL, "%s: h is given without a residual", who);
    Array ins[4], outs[6];
    int n_in = 0, n_out = 0;
    const int64_t live = rows > 0 ? 1 : 0;
    if ((rc = check_elements(x, rows, cols, ld_x, x_dtype, who, "x", &ins[n_in++])) ||
        (rc = check_elements(weight, live, cols, cols, w_dtype, who, "weight", &ins[n_in++])))
        return rc;
    if (residual &&
        (rc = check_elements(residual, rows, cols, ld_r, r_dtype, who, "residual", &ins[n_in++])))
        return rc;
    if (bias &&
        (rc = check_elements(bias, live, cols, cols, w_dtype, who, "bias", &ins[n_in++])))
        return rc;
    if (rows == 0) return ok();
    if (!h && !y && !q && !mean && !rstd) return fail(ZERO_EINVAL, "%s: no output is given", who);
    uint32_t same[6] = {};  // inputs that an output may be
    if (h) {
        if (same_array(h, r_dtype, ld_h, x, x_dtype, ld_x)) same[n_out] |= 1u;
        if (same_array(h, r_dtype, ld_h, residual, r_dtype, ld_r)) same[n_out] |= 4u;
        if ((rc = check_elements(h, rows, cols, ld_h, r_dtype, who, "h", &outs[n_out++])))
            return rc;
    }
    if (y) {
        if (same_array(y, y_dtype, ld_y, x, x_dtype, ld_x)) same[n_out] |= 1u;
        if ((rc = check_elements(y, rows, cols, ld_y, y_dtype, who, "y", &outs[n_out++])))
            return rc;
    }
    if (q) {
        if ((rc = check_q8(q, ld_q, s, ld_s, rows, cols, who, "q", "s", &outs[n_out],
                           &outs[n_out + 1])))
            return rc;
        n_out += 2;
    }
    if (mean && (rc = check_vector(mean, rows, who, "mean", &outs[n_out++]))) return rc;
    if (rstd && (rc = check_vector(rstd, rows, who, "rstd", &outs[n_out++]))) return rc;
    for (int o = 0; o < n_out; ++o)
        if ((rc = check_apart_but(outs[o], ins, n_in, same[o], who))) return rc;
    if ((rc = check_outputs(outs, n_out, who))) return rc;
    if (rows > kMaxGrid) return too_many(who);
    zero::LayerNormArgs a = {};
    a.x = x; a.res = residual; a.weight = weight; a.bias = bias;
    a.ld_x = ld_x; a.ld_r = ld_r; a.ld_h = ld_h; a.ld_y = ld_y; a.ld_q = ld_q; a.ld_s = ld_s;
    a.rows = rows;
    a.cols = static_cast<int32_t>(cols);
    a.x_dtype = x_dtype; a.r_dtype = r_dtype; a.w_dtype = w_dtype; a.y_dtype = y_dtype;
    a.fmt = fmt;
    a.eps = eps;
    a.h = h; a.y = y; a.q = static_cast<uint8_t*>(q); a.s = s; a.mean = mean; a.rstd = rstd;
    const hipError_t e = zero::launch_layernorm(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, who);
}

int64_t zero_layernorm_backward_workspace(int64_t rows, int64_t cols) {
    const char* who = "zero_layernorm_backward_workspace";
    if (check_size(rows, who, "rows") || check_layernorm_cols(cols, who)) return -1;
    ok();
    return 8 * cols * zero::layernorm_backward_parts(rows, static_cast<int32_t>(cols));
}

int zero_layernorm_backward(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* h,
                            int32_t h_dtype, int64_t ld_h, const void* weight, int32_t w_dtype,
                            const float* mean, const float* rstd, const void* dresidual,
                            int32_t dr_dtype, int64_t ld_dr, int64_t rows, int64_t cols, void* dx,
                            int32_t dx_dtype, int64_t ld_dx, void* dw, void* db, int32_t dw_dtype,
                            void* workspace, int64_t workspace_bytes, void* stream) {
    const char* who = "zero_layernorm_backward";
    int rc;
    if ((rc = check_size(rows, who, "rows")) || (rc = check_layernorm_cols(cols, who))) return rc;
    const int64_t live = rows > 0 ? 1 : 0;
    Array ins[6], outs[4];
    int n_in = 0, n_out = 0;
    if ((rc = check_elements(dy, rows, cols, ld_dy, dy_dtype, who, "dy", &ins[n_in++])) ||
        (rc = check_elements(h, rows, cols, ld_h, h_dtype, who, "h", &ins[n_in++])) ||
        (rc = check_elements(weight, live, cols, cols, w_dtype, who, "weight", &ins[n_in++])) ||
        (rc = check_vector(mean, rows, who, "mean", &ins[n_in++])) ||
        (rc = check_vector(rstd, rows, who, "rstd", &ins[n_in++])) ||
        (rc = check_elements(dx, rows, cols, ld_dx, dx_dtype, who, "dx", &outs[n_out++])))
        return rc;
    if (dresidual && (rc = check_elements(dresidual, rows, cols, ld_dr, dr_dtype, who, "dresidual",
                                          &ins[n_in++])))
        return rc;
    const int64_t parts = zero::layernorm_backward_parts(rows, static_cast<int32_t>(cols));
    if (dw || db) {
        if (dw && (rc = check_elements(dw, 1, cols, cols, dw_dtype, who, "dw", &outs[n_out++])))
            return rc;
        if (db && (rc = check_elements(db, 1, cols, cols, dw_dtype, who, "db", &outs[n_out++])))
            return rc;
        if (workspace_bytes < 8 * cols * parts)
            return fail(ZERO_ERANGE, "%s: workspace_bytes = %lld, %lld are needed", who,
                        static_cast<long long>(workspace_bytes),
                        static_cast<long long>(8 * cols * parts));
        if ((rc = check_array(workspace, 2 * parts, cols, cols, 4, 16, who, "workspace",
                              &outs[n_out++])))
            return rc;
    }
    uint32_t same = 0;
    if (same_array(dx, dx_dtype, ld_dx, dy, dy_dtype, ld_dy)) same |= 1u;
    if (same_array(dx, dx_dtype, ld_dx, h, h_dtype, ld_h)) same |= 2u;
    if (dresidual && same_array(dx, dx_dtype, ld_dx, dresidual, dr_dtype, ld_dr)) same |= 32u;
    for (int o = 0; o < n_out; ++o)
        if ((rc = check_apart_but(outs[o], ins, n_in, o == 0 ? same : 0u, who))) return rc;
    if ((rc = check_outputs(outs, n_out, who))) return rc;
    if (rows > kMaxGrid) return too_many(who);
    zero::LayerNormBackwardArgs a = {};
    a.dy = dy; a.h = h; a.weight = weight; a.dres = dresidual; a.mean = mean; a.rstd = rstd;
    a.ld_dy = ld_dy; a.ld_h = ld_h; a.ld_dr = ld_dr; a.ld_dx = ld_dx;
    a.rows = rows;
    a.cols = static_cast<int32_t>(cols);
    a.dy_dtype = dy_dtype; a.h_dtype = h_dtype; a.w_dtype = w_dtype; a.dr_dtype = dr_dtype;
    a.dx_dtype = dx_dtype; a.dw_dtype = dw_dtype;
    a.dx = dx; a.dw = dw; a.db = db;
    a.parts = dw || db ? static_cast<float*>(workspace) : nullptr;
    const hipError_t e = zero::launch_layernorm_backward(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, who);
}

int zero_act(const void* gate, int64_t ld_g, const void* up, int64_t ld_u, int32_t x_dtype,
             int32_t kind, int64_t rows, int64_t cols, void* y, int32_t y_dtype, int64_t ld_y,
             void* q, int32_t fmt, int64_t ld_q, uint8_t* s, int64_t ld_s, void* gate_q,
             int32_t ck_fmt, int64_t ld_gq, uint8_t* gate_s, int64_t ld_gs, void* up_q,
             int64_t ld_uq, uint8_t* up_s, int64_t ld_us, void* stream) {
    const char* who = "zero_act";
    int rc;
    if ((rc = check_dtype(x_dtype, who, "x_dtype")) || (rc = check_kind(kind, who)) ||
        (rc = check_size(rows, who, "rows")) || (rc = check_size(cols, who, "cols")))
        return rc;
    if (!q != !s) return fail(ZERO_EINVAL, "%s: q and s go together", who);
    if (!gate_q != !gate_s) return fail(ZERO_EINVAL, "%s: gate_q and gate_s go together", who);
    if (!up_q != !up_s) return fail(ZERO_EINVAL, "%s: up_q and up_s go together", who);
    if (q && (rc = check_fmt(fmt, who, "fmt"))) return rc;
    if ((gate_q || up_q) && (rc = check_fmt(ck_fmt, who, "ck_fmt"))) return rc;
    if (rows == 0 || cols == 0) return ok();
    if (up_q && !up) return fail(ZERO_EINVAL, "%s: up_q is given without an up", who);
    if (!y && !q && !gate_q && !up_q) return fail(ZERO_EINVAL, "%s: no output is given", who);
    Array ins[2], outs[7];
    int n_in = 0, n_out = 0;
    uint32_t same = 0;
    if ((rc = check_elements(gate, rows, cols, ld_g, x_dtype, who, "gate", &ins[n_in++])) ||
        (up && (rc = check_elements(up, rows, cols, ld_u, x_dtype, who, "up", &ins[n_in++]))))
        return rc;
    if (y) {
        if ((rc = check_elements(y, rows, cols, ld_y, y_dtype, who, "y", &outs[n_out++]))) return rc;
        if (same_array(y, y_dtype, ld_y, gate, x_dtype, ld_g)) same |= 1u;
        if (same_array(y, y_dtype, ld_y, up, x_dtype, ld_u)) same |= 2u;
    }
    if (q) {
        if ((rc = check_q8(q, ld_q, s, ld_s, rows, cols, who, "q", "s", &outs[n_out],
                           &outs[n_out + 1])))
            return rc;
        n_out += 2;
    }
    if (gate_q) {
        if ((rc = check_q8(gate_q, ld_gq, gate_s, ld_gs, rows, cols, who, "gate_q", "gate_s",
                           &outs[n_out], &outs[n_out + 1])))
            return rc;
        n_out += 2;
    }
    if (up_q) {
        if ((rc = check_q8(up_q, ld_uq, up_s, ld_us, rows, cols, who, "up_q", "up_s", &outs[n_out],
                           &outs[n_out + 1])))
            return rc;
        n_out += 2;
    }
    for (int o = 0; o < n_out; ++o)
        if ((rc = check_apart_but(outs[o], ins, n_in, y && o == 0 ? same : 0u, who))) return rc;
    if ((rc = check_outputs(outs, n_out, who))) return rc;
    if (zero::act_blocks(rows, cols) > kMaxGrid) return too_many(who);
    zero::ActArgs a = {};
    a.gate = gate; a.up = up;
    a.rows = rows; a.cols = cols;
    a.ld_g = ld_g; a.ld_u = ld_u; a.ld_y = ld_y; a.ld_q = ld_q; a.ld_s = ld_s;
    a.ld_gq = ld_gq; a.ld_gs = ld_gs; a.ld_uq = ld_uq; a.ld_us = ld_us;
    a.x_dtype = x_dtype; a.kind = kind; a.y_dtype = y_dtype; a.fmt = fmt; a.ck_fmt = ck_fmt;
    a.y = y;
    a.q = static_cast<uint8_t*>(q); a.s = s;
    a.gate_q = static_cast<uint8_t*>(gate_q); a.gate_s = gate_s;
    a.up_q = static_cast<uint8_t*>(up_q); a.up_s = up_s;
    const hipError_t e = zero::launch_act(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, who);
}

int zero_act_backward(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* gate_q,
                      int32_t ck_fmt, int64_t ld_gq, const uint8_t* gate_s, int64_t ld_gs,
                      const void* up_q, int64_t ld_uq, const uint8_t* up_s, int64_t ld_us,
                      int32_t kind, int64_t rows, int64_t cols, void* dgate, int64_t ld_dg,
                      void* dup, int64_t ld_du, int32_t dx_dtype, void* y, int32_t y_dtype,
                      int64_t ld_y, void* stream) {
    const char* who = "zero_act_backward";
    int rc;
    if ((rc = check_dtype(dy_dtype, who, "dy_dtype")) ||
        (rc = check_dtype(dx_dtype, who, "dx_dtype")) || (rc = check_fmt(ck_fmt, who, "ck_fmt")) ||
        (rc = check_kind(kind, who)) || (rc = check_size(rows, who, "rows")) ||
        (rc = check_size(cols, who, "cols")))
        return rc;
    if (!up_q != !up_s) return fail(ZERO_EINVAL, "%s: up_q and up_s go together", who);
    if (rows == 0 || cols == 0) return ok();
    if (!up_q != !dup) return fail(ZERO_EINVAL, "%s: dup goes with up_q", who);
    Array ins[5], outs[3];
    int n_in = 0, n_out = 0;
    if ((rc = check_elements(dy, rows, cols, ld_dy, dy_dtype, who, "dy", &ins[0])) ||
        (rc = check_q8(gate_q, ld_gq, gate_s, ld_gs, rows, cols, who, "gate_q", "gate_s", &ins[1],
                       &ins[2])))
        return rc;
    n_in = 3;
    if (up_q) {
        if ((rc = check_q8(up_q, ld_uq, up_s, ld_us, rows, cols, who, "up_q", "up_s", &ins[3],
                           &ins[4])))
            return rc;
        n_in = 5;
    }
    uint32_t same[3] = {};
    same[n_out] = same_array(dgate, dx_dtype, ld_dg, dy, dy_dtype, ld_dy);
    if ((rc = check_elements(dgate, rows, cols, ld_dg, dx_dtype, who, "dgate", &outs[n_out++])))
        return rc;
    if (dup) {
        same[n_out] = same_array(dup, dx_dtype, ld_du, dy, dy_dtype, ld_dy);
        if ((rc = check_elements(dup, rows, cols, ld_du, dx_dtype, who, "dup", &outs[n_out++])))
            return rc;
    }
    if (y) {
        same[n_out] = same_array(y, y_dtype, ld_y, dy, dy_dtype, ld_dy);
        if ((rc = check_elements(y, rows, cols, ld_y, y_dtype, who, "y", &outs[n_out++]))) return rc;
    }
    for (int o = 0; o < n_out; ++o)
        if ((rc = check_apart_but(outs[o], ins, n_in, same[o], who))) return rc;
    if ((rc = check_outputs(outs, n_out, who))) return rc;
    if (zero::act_blocks(rows, cols) > kMaxGrid) return too_many(who);
    zero::ActBackwardArgs a = {};
    a.dy = dy;
    a.gate_q = static_cast<const uint8_t*>(gate_q); a.gate_s = gate_s;
    a.up_q = static_cast<const uint8_t*>(up_q); a.up_s = up_s;
    a.rows = rows; a.cols = cols;
    a.ld_dy = ld_dy; a.ld_gq = ld_gq; a.ld_gs = ld_gs; a.ld_uq = ld_uq; a.ld_us = ld_us;
    a.ld_dg = ld_dg; a.ld_du = ld_du; a.ld_y = ld_y;
    a.dy_dtype = dy_dtype; a.ck_fmt = ck_fmt; a.kind = kind; a.dx_dtype = dx_dtype;
    a.y_dtype = y_dtype;
    a.dgate = dgate; a.dup = dup; a.y = y;
    const hipError_t e = zero::launch_act_backward(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, who);
}

int zero_logprob(const void* logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab,
                 const void* ids, int32_t id_bytes, float temperature, float* logp, float* entropy,
                 float* lse, int32_t* top_index, void* top_logit, int32_t top, int64_t ld_top,
                 void* stream) {
    const char* who = "zero_logprob";
    int rc;
    if ((rc = check_logprob_values(dtype, rows, vocab, ids, id_bytes, temperature, who))) return rc;
    if (!top_index != !top_logit)
        return fail(ZERO_EINVAL, "%s: top_index and top_logit go together", who);
    if (top_index && top < 1) return fail(ZERO_EINVAL, "%s: top = %d < 1", who, top);
    if (top_index && top > ZERO_LOGPROB_MAX_TOP)
        return fail(ZERO_ERANGE, "%s: top = %d is above %d", who, top, ZERO_LOGPROB_MAX_TOP);
    if (rows == 0) return ok();
    if (logp && !ids) return fail(ZERO_EINVAL, "%s: logp is given without ids", who);
    if (!logp && !entropy && !lse && !top_index)
        return fail(ZERO_EINVAL, "%s: no output is given", who);
    Array ins[2], outs[5];
    int n_in = 0, n_out = 0;
    if ((rc = check_logits(logits, dtype, ld, rows, vocab, ids, id_bytes, who, ins, &n_in)) ||
        (logp && (rc = check_vector(logp, rows, who, "logp", &outs[n_out++]))) ||
        (entropy && (rc = check_vector(entropy, rows, who, "entropy", &outs[n_out++]))) ||
        (lse && (rc = check_vector(lse, rows, who, "lse", &outs[n_out++]))))
        return rc;
    if (top_index &&
        ((rc = check_array(top_index, rows, top, ld_top, 4, 4, who, "top_index", &outs[n_out++])) ||
         (rc = check_elements(top_logit, rows, top, ld_top, dtype, who, "top_logit",
                              &outs[n_out++]))))
        return rc;
    for (int o = 0; o < n_out; ++o)
        if ((rc = check_apart_but(outs[o], ins, n_in, 0u, who))) return rc;
    if ((rc = check_outputs(outs, n_out, who))) return rc;
    if (rows > kMaxGrid) return too_many(who);
    zero::LogprobArgs a = {};
    a.logits = logits; a.ids = ids;
    a.rows = rows; a.vocab = vocab; a.ld = ld; a.ld_top = ld_top;
    a.dtype = dtype; a.id_bytes = id_bytes; a.top = top_index ? top : 0;
    a.tau = temperature;
    a.logp = logp; a.entropy = entropy; a.lse = lse;
    a.top_index = top_index; a.top_logit = top_logit;
    const hipError_t e = zero::launch_logprob(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, who);
}

int zero_logprob_backward(const void* logits, int32_t dtype, int64_t ld, int64_t rows,
                          int64_t vocab, const void* ids, int32_t id_bytes, float temperature,
                          const float* lse, const float* dlogp, const float* entropy,
                          const float* dentropy, float loss_scale, const zero_step_control* d_ctl,
                          void* grad, int64_t ld_grad, void* stream) {
    const char* who = "zero_logprob_backward";
    int rc;
    if ((rc = check_logprob_values(dtype, rows, vocab, ids, id_bytes, temperature, who))) return rc;
    if (d_ctl) {
        if ((rc = check_ctl(d_ctl, who))) return rc;
    } else if (!finite_f(loss_scale) || !(loss_scale > 0.0f)) {
        return fail(ZERO_EINVAL, "%s: loss_scale = %g is not finite and > 0", who,
                    static_cast<double>(loss_scale));
    }
    if (rows == 0) return ok();
    if (!dlogp && !dentropy) return fail(ZERO_EINVAL, "%s: neither dlogp nor dentropy is given", who);
    if (dlogp && !ids) return fail(ZERO_EINVAL, "%s: dlogp is given without ids", who);
    if (dentropy && !entropy)
        return fail(ZERO_EINVAL, "%s: dentropy is given without entropy", who);
    Array ins[6], out;
    int n_in = 0;
    if ((rc = check_logits(logits, dtype, ld, rows, vocab, ids, id_bytes, who, ins, &n_in)) ||
        (rc = check_vector(lse, rows, who, "lse", &ins[n_in++])) ||
        (dlogp && (rc = check_vector(dlogp, rows, who, "dlogp", &ins[n_in++]))) ||
        (dentropy && (rc = check_vector(entropy, rows, who, "entropy", &ins[n_in++]))) ||
        (dentropy && (rc = check_vector(dentropy, rows, who, "dentropy", &ins[n_in++]))) ||
        (rc = check_elements(grad, rows, vocab, ld_grad, dtype, who, "grad", &out)))
        return rc;
    const bool in_place = grad == logits;
    if (in_place && ld_grad != ld)
        return fail(ZERO_EINVAL, "%s: grad is the logits, with another row stride", who);
    if ((rc = check_apart_but(out, ins, n_in, in_place ? 1u : 0u, who))) return rc;
    if (rows > kMaxGrid || zero::logprob_backward_blocks(rows, vocab) > kMaxGrid)
        return too_many(who);
    zero::LogprobBackwardArgs a = {};
    a.logits = logits; a.ids = ids;
    a.rows = rows; a.vocab = vocab; a.ld = ld; a.ld_grad = ld_grad;
    a.dtype = dtype; a.id_bytes = id_bytes;
    a.tau = temperature; a.S = loss_scale;
    a.ctl = d_ctl;
    a.lse = lse; a.dlogp = dlogp; a.entropy = entropy; a.dentropy = dentropy;
    a.grad = grad;
    const hipError_t e = zero::launch_logprob_backward(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, who);
}

}  // extern "C"
