/*
 * zero_model.h -- C ABI of the operators at a language model's two ends and in
 * its feed-forward layers, on AMD Instinct MI355X (gfx950).  They run around
 * the products and norms of zero_train.h and before the shard step of
 * zero_step.h:
 *
 *   zero_embed       rows of a table by token, and the table's gradient, from
 *                    the tokens sorted by their row
 *   zero_layernorm   residual addition and layer norm, with an 8-bit output
 *                    for the next product; and its backward
 *   zero_act         (gated) activation that keeps its inputs as 8-bit
 *                    checkpoints; and its backward from those
 *   zero_logprob     log probability of a given token, entropy and the top
 *                    alternatives of each row of logits (the entries that
 *                    zero_distill takes from a teacher); and the gradient,
 *                    multiplied by the loss scale
 *
 * The conventions, element types, 8-bit block layout ("q8") and error codes are
 * those of zero_train.h: DEVICE pointers owned by the caller, work enqueued on
 * `stream`, every argument checked before anything is enqueued, no allocation,
 * no state kept between calls, fp32 arithmetic rounded once into the output's
 * type, the same bits from a repeated call.  Outputs overlap neither inputs nor
 * each other, apart from the cases named; arrays of one row stride may be
 * different column ranges of one matrix.  rows == 0 (tokens == 0) is a valid
 * call.  A workspace belongs to one call at a time: calls that may run at the
 * same time, replayed graphs too, need one each.
 */
#ifndef ZERO_MODEL_H
#define ZERO_MODEL_H

#include <stdint.h>

#include "zero_train.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZERO_EMBED_MAX_TOKENS 16777216 /* most tokens of the embedding's backward */
#define ZERO_LAYERNORM_MAX_COLS 65536  /* widest row of the layer norm calls      */
#define ZERO_LOGPROB_MAX_TOP 128       /* most alternatives per row               */

#define ZERO_SILU 0      /* f(g) = g / (1 + exp(-g))                              */
#define ZERO_GELU 1      /* f(g) = g Phi(g), Phi the normal distribution's        */
#define ZERO_GELU_TANH 2 /* f(g) = g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3)))  */

/*
 * zero_embed -- y[r] = scale * table[ids[r]].
 *
 *   table, t_dtype, ld_t   [vocab][cols], 1 <= vocab, cols <= 2^31 - 1
 *   ids, id_bytes          int32 (4) or int64 (8) [tokens], 0 <= tokens <= 2^31 - 1
 *   scale                  finite
 *   y, y_dtype, ld_y       [tokens][cols]
 * A negative id is padding: its row of y is zero.  A row whose id is vocab or
 * above is NaN, which ends up in the step's overflow check.  Returns ZERO_OK,
 * ZERO_EINVAL, ZERO_EALIGN or ZERO_EHIP.
 *
 * zero_embed_ctl -- the same from the copy of the fp16 parameters that a control
 * block says is current: tables_fp16[d_ctl->cur] (HOST array of two DEVICE
 * pointers), read on the device.
 */
int zero_embed(const void* table, int32_t t_dtype, int64_t vocab, int64_t cols, int64_t ld_t,
               const void* ids, int32_t id_bytes, int64_t tokens, float scale, void* y,
               int32_t y_dtype, int64_t ld_y, void* stream);
int zero_embed_ctl(const void* const* tables_fp16, int64_t vocab, int64_t cols, int64_t ld_t,
                   const void* ids, int32_t id_bytes, int64_t tokens, float scale, void* y,
                   int32_t y_dtype, int64_t ld_y, const zero_step_control* d_ctl, void* stream);

/* Bytes of workspace zero_embed_backward needs (HOST, synchronous): at most
 * 20 * tokens + (tokens + 64) * cols / 2 + 65536 of them; -1 with an error
 * text if the sizes are refused. */
int64_t zero_embed_backward_workspace(int64_t tokens, int64_t vocab, int64_t cols);

/*
 * zero_embed_backward -- dtable[v] = scale * sum of dy[r] over the tokens r with
 * ids[r] == v, added in fp32 in an order fixed by the ids and sizes, rounded
 * once.
 *
 *   dy, dy_dtype, ld_dy      [tokens][cols], 0 <= tokens <= ZERO_EMBED_MAX_TOKENS
 *   ids, id_bytes            [tokens]; tokens whose id is negative, vocab or above
 *                            add nothing
 *   dtable, dt_dtype, ld_dt  [vocab][cols]; may be a slot of a gradient bucket
 *   accumulate               0: every row is written, zeros where no token is;
 *                            1: the sum is added to the rows that have tokens (in
 *                            fp32, rounded once), the others are left alone
 *   workspace                16-byte aligned, workspace_bytes >= what
 *                            zero_embed_backward_workspace says
 * Returns ZERO_OK, ZERO_EINVAL, ZERO_EALIGN, ZERO_ERANGE (tokens,
 * workspace_bytes) or ZERO_EHIP.
 */
int zero_embed_backward(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* ids,
                        int32_t id_bytes, int64_t tokens, int64_t vocab, int64_t cols, float scale,
                        void* dtable, int32_t dt_dtype, int64_t ld_dt, int32_t accumulate,
                        void* workspace, int64_t workspace_bytes, void* stream);

/*
 * zero_layernorm -- residual addition and layer norm of each row:
 *   h = x + residual (or x), mean = mean(h), rstd = 1 / sqrt(mean((h - mean)^2) + eps),
 *   y = (h - mean) * rstd * weight + bias
 * with h kept in fp32 for the norm.
 *
 *   x, x_dtype, ld_x           [rows][cols], 0 <= rows <= 2^31 - 1,
 *                              1 <= cols <= ZERO_LAYERNORM_MAX_COLS
 *   residual, r_dtype, ld_r    [rows][cols], or NULL
 *   weight, bias, w_dtype      [cols] each, of one type; bias may be NULL: 0
 *   eps                        finite, >= 0
 *   h, ld_h                    [rows][cols] of r_dtype: h rounded; only with a
 *                              residual; NULL: not written; may be residual
 *                              itself (same ld), or x itself where the dtypes
 *                              agree (same ld)
 *   y, y_dtype, ld_y           [rows][cols], or NULL; may be x itself (same
 *                              dtype and ld)
 *   q, fmt, ld_q, s, ld_s      y, unrounded, in the q8 layout, or q and s NULL
 *   mean, rstd                 fp32[rows] each, or NULL
 * At least one output is given.  A row with a non-finite h is NaN throughout,
 * its mean and rstd what the formulas give; sums of squares are fp32's, as in
 * zero_rmsnorm.  Returns ZERO_OK, ZERO_EINVAL, ZERO_EALIGN, ZERO_ERANGE (cols)
 * or ZERO_EHIP.
 */
int zero_layernorm(const void* x, int32_t x_dtype, int64_t ld_x, const void* residual,
                   int32_t r_dtype, int64_t ld_r, const void* weight, const void* bias,
                   int32_t w_dtype, int64_t rows, int64_t cols, float eps, void* h, int64_t ld_h,
                   void* y, int32_t y_dtype, int64_t ld_y, void* q, int32_t fmt, int64_t ld_q,
                   uint8_t* s, int64_t ld_s, float* mean, float* rstd, void* stream);

/* Bytes of workspace zero_layernorm_backward needs for rows x cols (HOST,
 * synchronous): fp32 partial rows of dw and db, at most 8 * 1024 * cols bytes;
 * -1 with an error text if the sizes are refused. */
int64_t zero_layernorm_backward_workspace(int64_t rows, int64_t cols);

/*
 * zero_layernorm_backward -- the gradients of zero_layernorm.  With
 * xhat = (h - mean) * rstd and g = dy * weight:
 *   dx = dresidual (or 0) + rstd * (g - mean(g) - xhat * mean(g * xhat))
 *   dw = sum over rows of dy * xhat,   db = sum over rows of dy
 * dx is the gradient of both x and residual; dresidual is what arrives at h
 * from the rest of the residual stream.  The rows of dw and db are summed in
 * fp32 in an order fixed by the sizes.
 *
 *   dy, dy_dtype, ld_dy        [rows][cols], gradient of y
 *   h, h_dtype, ld_h           [rows][cols], as zero_layernorm left it
 *   weight, w_dtype            [cols]
 *   mean, rstd                 fp32[rows], as zero_layernorm left them
 *   dresidual, dr_dtype, ld_dr [rows][cols], or NULL
 *   dx, dx_dtype, ld_dx        [rows][cols]; may be dy, h or dresidual itself
 *                              (same dtype and ld)
 *   dw, db, dw_dtype           [cols] each, of one type; either may be NULL
 *   workspace                  16-byte aligned, workspace_bytes >= what
 *                              zero_layernorm_backward_workspace says; unused and
 *                              may be NULL if dw and db are NULL
 * rows == 0 gives dw = db = 0.  Returns ZERO_OK, ZERO_EINVAL, ZERO_EALIGN,
 * ZERO_ERANGE (cols, workspace_bytes) or ZERO_EHIP.
 */
int zero_layernorm_backward(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* h,
                            int32_t h_dtype, int64_t ld_h, const void* weight, int32_t w_dtype,
                            const float* mean, const float* rstd, const void* dresidual,
                            int32_t dr_dtype, int64_t ld_dr, int64_t rows, int64_t cols, void* dx,
                            int32_t dx_dtype, int64_t ld_dx, void* dw, void* db, int32_t dw_dtype,
                            void* workspace, int64_t workspace_bytes, void* stream);

/*
 * zero_act -- y = f(gate) * up, or f(gate) without an up, and 8-bit checkpoints
 * of gate and up for the backward pass: 1 + 1/128 bytes per element kept instead
 * of the element.
 *
 *   gate, up, x_dtype, ld_g, ld_u   [rows][cols] each, of one type; up may be
 *                                   NULL.  They may be column ranges of one
 *                                   product.  0 <= rows, 0 <= cols
 *   kind                            ZERO_SILU, ZERO_GELU or ZERO_GELU_TANH
 *   y, y_dtype, ld_y                [rows][cols], or NULL; may be gate or up
 *                                   itself (same dtype and ld)
 *   q, fmt, ld_q, s, ld_s           y, unrounded, in the q8 layout, or NULL
 *   gate_q, ck_fmt, ld_gq, gate_s, ld_gs   gate in the q8 layout, or NULL
 *   up_q, ld_uq, up_s, ld_us        up in the q8 layout (of ck_fmt), or NULL
 * The checkpoints are what zero_q8_quantize makes of gate and up, bit for bit;
 * y is of the elements themselves.  At least one output is given.  An infinite
 * gate gives the formula's limit where f's is infinite, else NaN.
 *
 * f comes from the hardware's exponential, whose argument is rounded.  For gates
 * above 0 it is off by a few 2^-24 of its value; for gates below 0 also by up to
 * 2^-24 |g| (SiLU), 2^-24 g^2 (GELU) or 5 * 2^-24 |2u| (its tanh form, u what the
 * tanh is of).  SiLU is 0 below -87.3, where f is under 1.1e-36.  Returns ZERO_OK,
 * ZERO_EINVAL, ZERO_EALIGN or ZERO_EHIP.
 */
int zero_act(const void* gate, int64_t ld_g, const void* up, int64_t ld_u, int32_t x_dtype,
             int32_t kind, int64_t rows, int64_t cols, void* y, int32_t y_dtype, int64_t ld_y,
             void* q, int32_t fmt, int64_t ld_q, uint8_t* s, int64_t ld_s, void* gate_q,
             int32_t ck_fmt, int64_t ld_gq, uint8_t* gate_s, int64_t ld_gs, void* up_q,
             int64_t ld_uq, uint8_t* up_s, int64_t ld_us, void* stream);

/*
 * zero_act_backward -- the gradients of zero_act from its checkpoints.  With g
 * and u the values that the checkpoints stand for (u = 1 without an up):
 *   dgate = dy * u * f'(g),   dup = dy * f(g),   y = f(g) * u
 *
 *   dy, dy_dtype, ld_dy             [rows][cols], gradient of y
 *   gate_q, ck_fmt, ld_gq, gate_s, ld_gs, up_q, ld_uq, up_s, ld_us
 *                                   as zero_act left them; up_q and up_s NULL
 *                                   for an activation without up
 *   dgate, dup, dx_dtype, ld_dg, ld_du   [rows][cols] each, of one type; dup goes
 *                                   with up; one of dgate, dup and y may be dy
 *                                   itself (same dtype and ld)
 *   y, y_dtype, ld_y                [rows][cols]: y once more, for the next
 *                                   product's weight gradient; or NULL
 * Returns ZERO_OK, ZERO_EINVAL, ZERO_EALIGN or ZERO_EHIP.
 */
int zero_act_backward(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* gate_q,
                      int32_t ck_fmt, int64_t ld_gq, const uint8_t* gate_s, int64_t ld_gs,
                      const void* up_q, int64_t ld_uq, const uint8_t* up_s, int64_t ld_us,
                      int32_t kind, int64_t rows, int64_t cols, void* dgate, int64_t ld_dg,
                      void* dup, int64_t ld_du, int32_t dx_dtype, void* y, int32_t y_dtype,
                      int64_t ld_y, void* stream);

/*
 * zero_logprob -- of each row of logits, with z = logits / temperature:
 *   lse = log sum over v of exp(z_v),   p_v = exp(z_v - lse)
 *   logp = z_id - lse,   entropy = -sum over v of p_v log p_v
 * and the `top` largest logits with their places, largest first, ties by the
 * lowest place.
 *
 *   logits, dtype, ld    [rows][vocab], 0 <= rows <= 2^31 - 1, 1 <= vocab <= 2^31 - 1
 *   ids, id_bytes        int32 or int64 [rows]; NULL: every row counts and there
 *                        is no logp
 *   temperature          > 0; it and log2(e) / it finite
 *   logp, entropy, lse   fp32[rows] each, or NULL; logp needs ids
 *   top_index, top_logit int32 and dtype [rows][top], row stride ld_top of both;
 *                        both NULL: not written (top is then not looked at)
 *   top                  1 .. ZERO_LOGPROB_MAX_TOP
 * At least one output is given.
 *   - A row with a negative id is left out: logp, entropy and lse 0, top_index -1
 *     and top_logit -inf, whatever its logits hold.
 *   - A logit of -inf is no alternative: places that are left over have
 *     top_index -1 and top_logit -inf (entries that zero_distill leaves out).
 *   - A row with an id >= vocab, a NaN or +inf among its logits, or no logit above
 *     -inf gives NaN for logp, entropy and lse, and NaN at place 0 for each
 *     alternative, which zero_distill turns into NaN.
 *   - An lse beyond fp32's range is infinite (logits / temperature of 3e38), logp and
 *     entropy are taken without it.  top_logit has no negative zeros.
 * The order of a row's sums follows from rows, vocab, dtype and the row's address
 * modulo 16, so that the same row among few and among many, or at another place, may
 * differ in its last bits.
 * Returns ZERO_OK, ZERO_EINVAL, ZERO_EALIGN, ZERO_ERANGE (top) or ZERO_EHIP.
 */
int zero_logprob(const void* logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab,
                 const void* ids, int32_t id_bytes, float temperature, float* logp, float* entropy,
                 float* lse, int32_t* top_index, void* top_logit, int32_t top, int64_t ld_top,
                 void* stream);

/*
 * zero_logprob_backward -- with a = dlogp and b = dentropy, the gradients that
 * arrive at each row's logp and entropy (either NULL: 0; not both):
 *   grad_v = S / temperature * (a * ([v = id] - p_v) - b * p_v * (log p_v + entropy))
 * from the lse and entropy that zero_logprob left for the same logits, ids and
 * temperature.  -1 / n as dlogp makes it the gradient of a cross-entropy over n
 * tokens.
 *
 *   logits .. temperature   as in zero_logprob; ids NULL only if dlogp is NULL
 *   lse                     fp32[rows]; p_v is taken from it, with the error that
 *                           zero_distill_backward names
 *   dlogp, dentropy         fp32[rows], finite
 *   entropy                 fp32[rows]; with dentropy, else not looked at
 *   loss_scale, d_ctl       S is loss_scale (finite, > 0), or, when d_ctl is not
 *                           NULL, d_ctl->scale, read on the device
 *   grad, ld_grad           [rows][vocab] of dtype; may be the logits (same ld)
 * A row with a negative id, or with a and b both 0, has a gradient of 0, whatever
 * its logits hold; otherwise an id >= vocab or an lse of NaN gives NaN
 * throughout.  Returns ZERO_OK, ZERO_EINVAL, ZERO_EALIGN or ZERO_EHIP.
 */
int zero_logprob_backward(const void* logits, int32_t dtype, int64_t ld, int64_t rows,
                          int64_t vocab, const void* ids, int32_t id_bytes, float temperature,
                          const float* lse, const float* dlogp, const float* entropy,
                          const float* dentropy, float loss_scale, const zero_step_control* d_ctl,
                          void* grad, int64_t ld_grad, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_MODEL_H */
