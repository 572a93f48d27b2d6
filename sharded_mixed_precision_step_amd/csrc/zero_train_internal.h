// Internal interface between the host layer of the training operators
// (zero_train_abi.cpp) and their gfx950 kernels (zero_norm.hip, zero_q8.hip,
// zero_q8_gemm.hip, zero_distill.hip).  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_train.h"

namespace zero {

// HIP launches fewer than 2^32 lanes along a dimension.  Workgroups 0 ..
// blocks - 1 of `lanes` lanes each, in as many launches as that takes:
// launch(first, n) launches n of them from `first` on.
template <class Launch>
inline hipError_t in_launches(int64_t blocks, int64_t lanes, Launch launch) {
    const int64_t most = 0xffffffff / lanes;
    for (int64_t first = 0; first < blocks; first += most) {
        const int64_t left = blocks - first;
        const hipError_t e = launch(first, static_cast<uint32_t>(left < most ? left : most));
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

struct QuantizeArgs {
    const void* src[2];               // the copy cur picks; src[0] without a control block
    const zero_step_control* ctl;     // or NULL
    int64_t rows, cols, ld_src;
    uint8_t *q, *s, *qt, *st;
    int64_t ld_q, ld_s, ld_qt, ld_st;
    int32_t dtype, fmt;
};
int64_t quantize_blocks(int64_t rows, int64_t cols);  // workgroups of one call
hipError_t launch_q8_quantize(const QuantizeArgs& a, hipStream_t stream);

struct GemmArgs {
    const uint8_t *a, *sa, *b, *sb;
    int64_t ld_a, ld_sa, ld_b, ld_sb;
    int64_t m, n;
    int32_t kblocks;                  // blocks of 128 columns
    int32_t fmt_a, fmt_b, c_dtype, accumulate;
    void* c;
    int64_t ld_c;
};
int64_t gemm_tiles(int64_t m, int64_t n);
hipError_t launch_q8_gemm(const GemmArgs& a, hipStream_t stream);

struct NormArgs {
    const void *x, *res, *weight;
    int64_t ld_x, ld_r, ld_h, ld_y, ld_q, ld_s;
    int64_t rows;
    int32_t cols, x_dtype, r_dtype, w_dtype, y_dtype, fmt;
    float eps;
    void *h, *y;
    uint8_t *q, *s;
    float* rstd;
};
hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t stream);

struct NormBackwardArgs {
    const void *dy, *h, *weight, *dres;
    const float* rstd;
    int64_t ld_dy, ld_h, ld_dr, ld_dx;
    int64_t rows;
    int32_t cols, dy_dtype, h_dtype, w_dtype, dr_dtype, dx_dtype, dw_dtype;
    void *dx, *dw;
    float* parts;                     // [norm_backward_parts][cols]
};
int32_t norm_backward_parts(int64_t rows, int32_t cols);  // partial rows of dw
hipError_t launch_rmsnorm_backward(const NormBackwardArgs& a, hipStream_t stream);

struct DistillArgs {
    const void *logits, *index, *top_logit;
    const float* weight;
    int64_t rows, vocab, ld, ld_top;
    int32_t dtype, top_dtype, index_bytes, top;
    float tau;
    float S;
    const zero_step_control* ctl;     // S = ctl->scale when given
    float* loss;
    float* lse;                       // written by the forward and the fused call
    const float* lse_in;              // read by the backward
    void* grad;
    int64_t ld_grad;
};
enum DistillMode { kDistillForward, kDistillBackward, kDistillBoth };
hipError_t launch_distill(const DistillArgs& a, DistillMode mode, hipStream_t stream);

}  // namespace zero
