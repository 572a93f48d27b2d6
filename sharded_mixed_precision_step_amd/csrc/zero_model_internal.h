// Internal interface between the host layer of zero_model.h's operators
// (zero_model_abi.cpp) and their gfx950 kernels (zero_embed.hip,
// zero_layernorm.hip, zero_layernorm_backward.hip, zero_act.hip,
// zero_logprob.hip).  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_model.h"
#include "zero_train_internal.h"

namespace zero {

struct EmbedArgs {
    const void* table[2];          // the copy cur picks; table[0] without a control block
    const zero_step_control* ctl;  // or NULL
    const void* ids;
    int64_t tokens, vocab, cols, ld_t, ld_y;
    int32_t id_bytes, t_dtype, y_dtype;
    float scale;
    void* y;
};
int64_t embed_blocks(int64_t tokens, int64_t cols);  // workgroups of one call
hipError_t launch_embed(const EmbedArgs& a, hipStream_t stream);

// The backward's workspace: sorted keys and places twice (the passes of the
// sort go back and forth), digit counts of the sort's blocks, partial rows.
struct EmbedWorkspace {
    int64_t keys[2], order[2], counts, parts, bytes;  // byte offsets; total
};
EmbedWorkspace embed_workspace(int64_t tokens, int64_t cols);
struct EmbedBackwardArgs {
    const void *dy, *ids;
    int64_t tokens, vocab, cols, ld_dy, ld_dt;
    int32_t id_bytes, dy_dtype, dt_dtype, accumulate;
    float scale;
    void* dtable;
    char* workspace;               // embed_workspace(tokens, cols).bytes
};
// Workgroups of the largest of a call's launches.
int64_t embed_backward_blocks(int64_t tokens, int64_t vocab, int64_t cols, int64_t ld_dt,
                              int32_t dt_dtype);
hipError_t launch_embed_backward(const EmbedBackwardArgs& a, hipStream_t stream);

struct LayerNormArgs {
    const void *x, *res, *weight, *bias;
    int64_t ld_x, ld_r, ld_h, ld_y, ld_q, ld_s;
    int64_t rows;
    int32_t cols, x_dtype, r_dtype, w_dtype, y_dtype, fmt;
    float eps;
    void *h, *y;
    uint8_t *q, *s;
    float *mean, *rstd;
};
hipError_t launch_layernorm(const LayerNormArgs& a, hipStream_t stream);

struct LayerNormBackwardArgs {
    const void *dy, *h, *weight, *dres;
    const float *mean, *rstd;
    int64_t ld_dy, ld_h, ld_dr, ld_dx;
    int64_t rows;
    int32_t cols, dy_dtype, h_dtype, w_dtype, dr_dtype, dx_dtype, dw_dtype;
    void *dx, *dw, *db;
    float* parts;                  // [2][layernorm_backward_parts][cols], or NULL
};
int32_t layernorm_backward_parts(int64_t rows, int32_t cols);  // partial rows of dw, and of db
hipError_t launch_layernorm_backward(const LayerNormBackwardArgs& a, hipStream_t stream);

struct ActArgs {
    const void *gate, *up;
    int64_t rows, cols, ld_g, ld_u, ld_y, ld_q, ld_s, ld_gq, ld_gs, ld_uq, ld_us;
    int32_t x_dtype, kind, y_dtype, fmt, ck_fmt;
    void* y;
    uint8_t *q, *s, *gate_q, *gate_s, *up_q, *up_s;
};
int64_t act_blocks(int64_t rows, int64_t cols);  // workgroups of one call, either direction
hipError_t launch_act(const ActArgs& a, hipStream_t stream);

struct ActBackwardArgs {
    const void* dy;
    const uint8_t *gate_q, *gate_s, *up_q, *up_s;
    int64_t rows, cols, ld_dy, ld_gq, ld_gs, ld_uq, ld_us, ld_dg, ld_du, ld_y;
    int32_t dy_dtype, ck_fmt, kind, dx_dtype, y_dtype;
    void *dgate, *dup, *y;
};
hipError_t launch_act_backward(const ActBackwardArgs& a, hipStream_t stream);

struct LogprobArgs {
    const void *logits, *ids;
    int64_t rows, vocab, ld, ld_top;
    int32_t dtype, id_bytes, top;
    float tau;
    float *logp, *entropy, *lse;
    int32_t* top_index;
    void* top_logit;
};
hipError_t launch_logprob(const LogprobArgs& a, hipStream_t stream);

struct LogprobBackwardArgs {
    const void *logits, *ids;
    int64_t rows, vocab, ld, ld_grad;
    int32_t dtype, id_bytes;
    float tau, S;
    const zero_step_control* ctl;  // S = ctl->scale when given
    const float *lse, *dlogp, *entropy, *dentropy;
    void* grad;
};
int64_t logprob_backward_blocks(int64_t rows, int64_t vocab);
hipError_t launch_logprob_backward(const LogprobBackwardArgs& a, hipStream_t stream);

}  // namespace zero
