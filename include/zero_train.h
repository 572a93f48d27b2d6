/*
 * zero_train.h -- C ABI of the training operators that run right before and
 * right after the shard step of zero_step.h, on AMD Instinct MI355X (gfx950).
 *
 * The shard step takes loss-scaled fp16 gradients and leaves fp16 parameters.
 * These calls are the mixed-precision numerics on either side of it:
 *
 *   zero_q8_quantize   a matrix to 8 bits with a scale for each block of 128
 *                      (the parameters a step has just written, gradients)
 *   zero_q8_gemm       the matrix product of two such matrices (forward, input
 *                      gradient, weight gradient)
 *   zero_rmsnorm       residual addition and root-mean-square norm, with an
 *                      8-bit output for the next product; and its backward
 *   zero_distill       distillation loss from a teacher's top logits, and its
 *                      gradient multiplied by the loss scale
 *
 * The conventions are those of zero_step.h: DEVICE pointers owned by the
 * caller unless marked HOST, work enqueued on `stream`, every argument checked
 * before anything is enqueued, no allocation, no state kept between calls,
 * zero_last_error_string() for the text of an error.  Results do not depend on
 * timing: no call uses floating-point atomics, so a call repeated on the same
 * inputs gives the same bits.
 *
 * Element types (dtype arguments): ZERO_F32, ZERO_F16 (IEEE binary16),
 * ZERO_BF16.  A pointer to elements is aligned to its element; strides ("ld")
 * count elements between the starts of consecutive rows, and a row's elements
 * are contiguous.  Values are taken to fp32 exactly, computed in fp32 and
 * rounded once, to nearest even, into the output's type; a value beyond an
 * fp16 output's range becomes inf, which zero_overflow_check then sees.
 * Overlap is judged from an array's first byte to its last, the gaps between
 * strided rows included.
 *
 * The 8-bit block layout ("q8").  A matrix of rows x cols is held as
 *   data    [rows][ld] 8-bit floats, ZERO_E4M3 (largest value 448, no inf) or
 *           ZERO_E5M2 (largest value 57344): ld >= P = cols rounded up to 128;
 *           the bytes of columns cols .. P-1 are zero.  16-byte aligned, ld a
 *           multiple of 16.
 *   scales  [rows][ld_s] bytes: byte b of a row holds e + 127 (E8M0), the scale
 *           2^e of columns 128b .. 128b+127; ld_s >= Q = P / 128 rounded up to
 *           4, and the bytes of blocks P/128 .. Q-1 are 127 (a scale of 1).
 *           4-byte aligned, ld_s a multiple of 4.
 * The value of an element is data * 2^e.  A block's scale is the smallest
 * power of two that brings the block's largest magnitude to the type's largest
 * value or below, so that nothing saturates and scaling is exact; e is held
 * to [-127, 127]; a block of zeros has scale 1.  A block with an inf or a NaN
 * has scale byte 255 (NaN) and NaN elements, padding included, so that every
 * product it enters is NaN and the overflow check of the step sees it.
 * Power-of-two scales are what gfx950's matrix cores apply themselves.
 */
#ifndef ZERO_TRAIN_H
#define ZERO_TRAIN_H

#include <stdint.h>

#include "zero_step.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZERO_F32 0
#define ZERO_F16 1
#define ZERO_BF16 2

#define ZERO_E4M3 0
#define ZERO_E5M2 1

#define ZERO_Q8_BLOCK 128
#define ZERO_Q8_MAX_LD 8388608    /* largest k and row stride of the product     */
#define ZERO_NORM_MAX_COLS 65536  /* widest row of the norm calls               */
#define ZERO_NORM_MAX_PARTS 1024  /* most partial rows of the norm's backward   */
#define ZERO_DISTILL_MAX_TOP 1024 /* most teacher entries per row               */

/*
 * zero_q8_quantize -- src [rows][cols] in the q8 layout, by rows, transposed,
 * or both in one pass over src.
 *
 *   src, dtype, ld_src   the matrix; ld_src >= cols
 *   fmt                  ZERO_E4M3 or ZERO_E5M2, of both outputs
 *   q, ld_q, s, ld_s     src in the q8 layout (blocks of 128 along a row); q and
 *                        s both NULL: not written
 *   qt, ld_qt, st, ld_st src transposed, [cols][rows], in the q8 layout (blocks
 *                        of 128 along a column of src); both NULL: not written
 * At least one output is given.  Outputs must not overlap src or each other.
 * rows == 0 or cols == 0 is a valid call that writes what the layout then holds:
 * nothing.  Returns ZERO_OK, ZERO_EINVAL (also for more than 2^31 - 1 tiles of
 * 128 x 128), ZERO_EALIGN or ZERO_EHIP.
 */
int zero_q8_quantize(const void* src, int32_t dtype, int64_t rows, int64_t cols, int64_t ld_src,
                     int32_t fmt, void* q, int64_t ld_q, uint8_t* s, int64_t ld_s, void* qt,
                     int64_t ld_qt, uint8_t* st, int64_t ld_st, void* stream);

/*
 * zero_q8_quantize_ctl -- zero_q8_quantize of fp16 parameters, from the copy
 * that a control block says is current: src is srcs_fp16[d_ctl->cur] (HOST
 * array of two DEVICE pointers, as the single-pass calls take them).  Enqueued
 * after zero_control_decide it quantizes the parameters the step has just
 * committed, or the previous ones if the step was skipped, with no read-back.
 */
int zero_q8_quantize_ctl(const void* const* srcs_fp16, int64_t rows, int64_t cols, int64_t ld_src,
                         int32_t fmt, void* q, int64_t ld_q, uint8_t* s, int64_t ld_s, void* qt,
                         int64_t ld_qt, uint8_t* st, int64_t ld_st,
                         const zero_step_control* d_ctl, void* stream);

/*
 * zero_q8_gemm -- c = a b^T of two q8 matrices: c[i][j] = sum over k of
 * a[i][k] * b[j][k].  Sums are fp32's where m <= 16 and n <= 8192.  Beyond that
 * they are those of gfx950's 8-bit matrix instructions: each eight neighbouring
 * products are added on a grid of 2^-13 of the largest one's power of two,
 * truncated towards zero; everything else is fp32.
 *
 *   a, fmt_a, ld_a, sa, ld_sa   q8 matrix [m][k]
 *   b, fmt_b, ld_b, sb, ld_sb   q8 matrix [n][k]
 *   k             columns of a and b; their padding up to a multiple of 128 is
 *                 read too and has to be zeros, as zero_q8_quantize leaves it
 *   c, c_dtype, ld_c   [m][n], ld_c >= n; rows may be a slot of a gradient bucket
 *   accumulate    0: c is written; 1: the product is added to c (the sum taken
 *                 in fp32 and rounded once)
 * With x [t][k], w [n][k] and dy [t][n] the products of a linear layer are
 * y = x w^T (a = x, b = w), dx = dy w (a = dy, b = w transposed) and
 * dw = dy^T x (a = dy transposed, b = x transposed).  k == 0 gives zeros,
 * whatever a, b, their scales and strides are.  c must not overlap a, b or their
 * scales.  Returns ZERO_OK, ZERO_EINVAL, ZERO_EALIGN, ZERO_ERANGE (k or a row
 * stride above ZERO_Q8_MAX_LD) or ZERO_EHIP; ZERO_EINVAL also for a c of more
 * than 2^27 tiles of 64 x 64.
 */
int zero_q8_gemm(const void* a, int32_t fmt_a, int64_t ld_a, const uint8_t* sa, int64_t ld_sa,
                 const void* b, int32_t fmt_b, int64_t ld_b, const uint8_t* sb, int64_t ld_sb,
                 int64_t m, int64_t n, int64_t k, void* c, int32_t c_dtype, int64_t ld_c,
                 int32_t accumulate, void* stream);

/*
 * zero_rmsnorm -- residual addition and root-mean-square norm of each row:
 *   h = x + residual (or x), rstd = 1 / sqrt(mean(h^2) + eps),
 *   y = h * rstd * weight
 * with h kept in fp32 for the norm.
 *
 *   x, x_dtype, ld_x           [rows][cols], 0 <= rows <= 2^31 - 1,
 *                              1 <= cols <= ZERO_NORM_MAX_COLS
 *   residual, r_dtype, ld_r    [rows][cols], or NULL
 *   weight, w_dtype            [cols]
 *   eps                        finite, >= 0
 *   h, ld_h                    [rows][cols] of r_dtype: h rounded; only with a
 *                              residual; NULL: not written; may be residual
 *                              itself (same ld), or x itself where the dtypes
 *                              agree (same ld)
 *   y, y_dtype, ld_y           [rows][cols], or NULL; may be x itself (same
 *                              dtype and ld)
 *   q, fmt, ld_q, s, ld_s      y, unrounded, in the q8 layout, or q and s NULL
 *   rstd                       fp32[rows], or NULL
 * At least one of h, y, q and rstd is given.  Apart from the cases named, no
 * output may overlap an input or another output.  A row with a non-finite h
 * gives NaN, or inf, where the formula does; sums of squares are fp32's, so
 * that rows beyond 1.8e19, which no fp16 row is, count as infinitely long and
 * squares of values below 1e-19 lose places, and below 2e-23 are zero (with
 * eps == 0 such rows have an rstd of inf).
 * rows == 0 is a no-op.  Returns ZERO_OK, ZERO_EINVAL, ZERO_EALIGN, ZERO_ERANGE
 * (cols) or ZERO_EHIP.
 */
int zero_rmsnorm(const void* x, int32_t x_dtype, int64_t ld_x, const void* residual,
                 int32_t r_dtype, int64_t ld_r, const void* weight, int32_t w_dtype, int64_t rows,
                 int64_t cols, float eps, void* h, int64_t ld_h, void* y, int32_t y_dtype,
                 int64_t ld_y, void* q, int32_t fmt, int64_t ld_q, uint8_t* s, int64_t ld_s,
                 float* rstd, void* stream);

/* Bytes of workspace zero_rmsnorm_backward needs for rows x cols (HOST,
 * synchronous): fp32 partial rows, at most ZERO_NORM_MAX_PARTS of them; -1
 * with an error text if the sizes are refused. */
int64_t zero_rmsnorm_backward_workspace(int64_t rows, int64_t cols);

/*
 * zero_rmsnorm_backward -- the gradients of zero_rmsnorm.  With xhat = h * rstd
 * and g = dy * weight:
 *   dx = dresidual (or 0) + rstd * (g - xhat * mean(g * xhat))
 *   dw = sum over rows of dy * xhat
 * dx is the gradient of both x and residual; dresidual is what arrives at h
 * from the rest of the residual stream.  dw's rows are summed in fp32 in an
 * order fixed by the sizes.
 *
 *   dy, dy_dtype, ld_dy        [rows][cols], gradient of y
 *   h, h_dtype, ld_h           [rows][cols], as zero_rmsnorm left it
 *   weight, w_dtype            [cols]
 *   rstd                       fp32[rows], as zero_rmsnorm left it
 *   dresidual, dr_dtype, ld_dr [rows][cols], or NULL
 *   dx, dx_dtype, ld_dx        [rows][cols]; may be dy, h or dresidual itself
 *                              (same dtype and ld)
 *   dw, dw_dtype               [cols], or NULL
 *   workspace                  16-byte aligned, workspace_bytes >= what
 *                              zero_rmsnorm_backward_workspace says; unused and
 *                              may be NULL if dw is NULL.  Calls that may run at
 *                              the same time, replayed graphs too, need one each
 * rows == 0 gives dw = 0.  Returns ZERO_OK, ZERO_EINVAL, ZERO_EALIGN,
 * ZERO_ERANGE (cols, workspace_bytes) or ZERO_EHIP.
 */
int zero_rmsnorm_backward(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* h,
                          int32_t h_dtype, int64_t ld_h, const void* weight, int32_t w_dtype,
                          const float* rstd, const void* dresidual, int32_t dr_dtype,
                          int64_t ld_dr, int64_t rows, int64_t cols, void* dx, int32_t dx_dtype,
                          int64_t ld_dx, void* dw, int32_t dw_dtype, void* workspace,
                          int64_t workspace_bytes, void* stream);

/* What the distillation calls read.  HOST struct.
 *
 * For each row r, with z = logits[r] / temperature over the vocab and
 * t = top_logit[r] / temperature over the row's entries: entry j says that the
 * teacher gave vocab index i_j the logit t_j; an entry with a negative index
 * is left out (a row with fewer entries is padded with -1).
 *   lse  = log sum over v of exp(z_v)              q_v = exp(z_v - lse)
 *   p_j  = exp(t_j) / sum over entries of exp(t)   (the teacher's top entries,
 *                                                  renormalized)
 *   loss = w * temperature^2 * sum_j p_j * (log p_j - log q_{i_j})
 *   gradient of z_v's logit = S * w * temperature *
 *                             (q_v - sum of p_j over entries with i_j = v)
 * with w = row_weight[r] (the caller's mask and mean) and S the loss scale.  An
 * index that comes twice counts twice.  An entry with p_j = 0 (a logit of
 * -inf) adds nothing, whatever q is there.
 *   - A row of weight 0 gives loss 0, lse 0 and gradient 0, whatever its
 *     logits and entries hold.
 *   - A row with no entry left (all negative indices, or logits of -inf) gives
 *     loss 0 and gradient 0.
 *   - A row with an index >= vocab, a NaN or +inf among its entries, a NaN or
 *     +inf among its logits, or no logit above -inf gives a loss and a gradient
 *     of NaN throughout, which the step's overflow check turns into a skip;
 *     lse is then NaN too.
 */
typedef struct zero_distill_inputs {
    const void* logits;      /* student logits [rows][vocab]                     */
    const void* top_index;   /* int32 or int64 [rows][top]                       */
    const void* top_logit;   /* [rows][top]                                      */
    const float* row_weight; /* fp32[rows], finite, or NULL: every weight is 1   */
    int64_t rows;            /* 0 .. 2^31 - 1                                    */
    int64_t vocab;           /* 1 .. 2^31 - 1                                    */
    int64_t ld_logits;       /* >= vocab                                         */
    int64_t ld_top;          /* >= top, of both top_index and top_logit          */
    int32_t logits_dtype;    /* ZERO_F32, ZERO_F16 or ZERO_BF16                  */
    int32_t top_dtype;       /* of top_logit                                     */
    int32_t index_bytes;     /* 4 or 8                                           */
    int32_t top;             /* entries per row, 1 .. ZERO_DISTILL_MAX_TOP       */
    float temperature;       /* > 0; it, its square and log2(e) / it finite      */
    int32_t pad_;
} zero_distill_inputs;

/*
 * zero_distill_forward -- loss fp32[rows] and lse fp32[rows] (either NULL: not
 * written; not both), reading the logits once.
 *
 * zero_distill_backward -- the gradient, in grad [rows][vocab] of
 * logits_dtype with row stride ld_grad >= vocab, from the lse that
 * zero_distill_forward left for the same inputs.  A different row_weight may
 * be given here, for instance the weight times a gradient that arrives at each
 * row's loss (for a row whose lse was taken with weight 0, only 0).  q_v is
 * taken from lse, which fp32 holds to 2^-24 of its size: logits / temperature of
 * magnitude Z put an error of Z * 2^-23 on q_v, and a row whose logits /
 * temperature all lie beyond fp32 has no such lse (zero_distill has none of
 * this).  grad may be the logits themselves (same ld).  S is loss_scale, or, when d_ctl is not NULL,
 * d_ctl->scale, the scale of the control block's next step, read on the
 * device; loss_scale is then not used.
 *
 * zero_distill -- both at once: loss, lse (either may be NULL) and grad.
 *
 * Outputs must not overlap the inputs (apart from grad = logits) or each
 * other.  loss_scale is finite and > 0.  rows == 0 is a no-op.  Return ZERO_OK,
 * ZERO_EINVAL, ZERO_EALIGN, ZERO_ERANGE (top) or ZERO_EHIP.
 */
int zero_distill_forward(const zero_distill_inputs* in, float* loss, float* lse, void* stream);
int zero_distill_backward(const zero_distill_inputs* in, const float* lse, float loss_scale,
                          const zero_step_control* d_ctl, void* grad, int64_t ld_grad,
                          void* stream);
int zero_distill(const zero_distill_inputs* in, float loss_scale, const zero_step_control* d_ctl,
                 float* loss, float* lse, void* grad, int64_t ld_grad, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_TRAIN_H */
