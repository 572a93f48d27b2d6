// Gradients of the root-mean-square norm.
//
// One pass over its arrays, bound by HBM, with the forward's row layout (one
// workgroup per row, eight elements per lane and step).
#include "zero_device.h"
#include "zero_train_internal.h"

namespace zero {
namespace {

using namespace dev;

// A workgroup takes rows blockIdx.x, + gridDim.x, ...; its lanes
// keep the same columns for every row, so dw's sum over those rows stays in
// registers and leaves once, as one fp32 partial row.
template <int T, int P, int DB, int HB, int RB>
__global__ __launch_bounds__(T) void rmsnorm_backward_kernel(const NormBackwardArgs a) {
    __shared__ float part[2][T / 64];
    const int t = threadIdx.x;
    float dw[P][8];
    float w[P][8];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * T + t) * 8;
        if (a.w_dtype == ZERO_F32) {
            const Raw8<4> r = load8<4>(a.weight, c, a.cols - c);
            widen8<4>(r, false, w[i]);
        } else {
            const Raw8<2> r = load8<2>(a.weight, c, a.cols - c);
            widen8<2>(r, a.w_dtype == ZERO_BF16, w[i]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) dw[i][k] = 0.0f;
    }
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        Raw8<DB> rd[P];
        Raw8<HB> rh[P];
        Raw8<RB == 0 ? 2 : RB> rr[P];
        const float rstd = a.rstd[row];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * T + t) * 8;
            rd[i] = load8<DB>(a.dy, row * a.ld_dy + c, a.cols - c);
            rh[i] = load8<HB>(a.h, row * a.ld_h + c, a.cols - c);
            if constexpr (RB != 0) rr[i] = load8<RB>(a.dres, row * a.ld_dr + c, a.cols - c);
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float d[8], h[8];
            widen8<DB>(rd[i], a.dy_dtype == ZERO_BF16, d);
            widen8<HB>(rh[i], a.h_dtype == ZERO_BF16, h);
            const int left = a.cols - (i * T + t) * 8;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float xhat = h[k] * rstd;
                // lanes behind the row's end hold zeros, which a non-finite
                // rstd would make NaN
                if (k < left) {
                    dot = __builtin_fmaf(d[k] * w[i][k], xhat, dot);
                    dw[i][k] = __builtin_fmaf(d[k], xhat, dw[i][k]);
                }
            }
        }
        const float mean = block_sum<T>(dot, part[flip]) / static_cast<float>(a.cols);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * T + t) * 8;
            float d[8], h[8], r[8];
            widen8<DB>(rd[i], a.dy_dtype == ZERO_BF16, d);
            widen8<HB>(rh[i], a.h_dtype == ZERO_BF16, h);
            if constexpr (RB != 0) widen8<RB>(rr[i], a.dr_dtype == ZERO_BF16, r);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float xhat = h[k] * rstd;
                const float inner = __builtin_fmaf(-xhat, mean, d[k] * w[i][k]);
                if constexpr (RB != 0) d[k] = __builtin_fmaf(rstd, inner, r[k]);
                else d[k] = rstd * inner;
            }
            store8(a.dx, row * a.ld_dx + c, a.cols - c, a.dx_dtype, d);
        }
    }
    if (!a.parts) return;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * T + t) * 8;
        store8(a.parts, static_cast<int64_t>(blockIdx.x) * a.cols + c, a.cols - c, ZERO_F32,
               dw[i]);
    }
}

// dw = the partial rows' sum: 64 columns per workgroup, 16 groups of lanes
// over the partial rows, then over the groups, in a fixed order.
constexpr int kDwCols = 64;
constexpr int kDwGroups = 16;
__global__ __launch_bounds__(kDwCols* kDwGroups) void rmsnorm_dw_kernel(const float* parts,
                                                                       int n_parts, int cols,
                                                                       void* dw, int dtype) {
    __shared__ float sums[kDwGroups][kDwCols];
    const int lane = threadIdx.x % kDwCols, group = threadIdx.x / kDwCols;
    const int c = blockIdx.x * kDwCols + lane;
    float v = 0.0f;
    if (c < cols) {
        int p = group;
        for (; p + 7 * kDwGroups < n_parts; p += 8 * kDwGroups) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = parts[static_cast<int64_t>(p + k * kDwGroups) * cols + c];
#pragma unroll
            for (int k = 0; k < 8; ++k) v += x[k];
        }
        for (; p < n_parts; p += kDwGroups) v += parts[static_cast<int64_t>(p) * cols + c];
    }
    sums[group][lane] = v;
    __syncthreads();
    if (group == 0 && c < cols) {
#pragma unroll
        for (int g = 1; g < kDwGroups; ++g) v += sums[g][lane];
        store1(dw, c, dtype, v);
    }
}

template <int T, int P, int DB, int HB>
void backward_types(const NormBackwardArgs& a, dim3 grid, hipStream_t stream) {
    if (!a.dres) rmsnorm_backward_kernel<T, P, DB, HB, 0><<<grid, T, 0, stream>>>(a);
    else if (a.dr_dtype == ZERO_F32)
        rmsnorm_backward_kernel<T, P, DB, HB, 4><<<grid, T, 0, stream>>>(a);
    else rmsnorm_backward_kernel<T, P, DB, HB, 2><<<grid, T, 0, stream>>>(a);
}

template <int T, int P>
void backward_shape(const NormBackwardArgs& a, dim3 grid, hipStream_t stream) {
    const bool d4 = a.dy_dtype == ZERO_F32, h4 = a.h_dtype == ZERO_F32;
    if (d4) {
        if (h4) backward_types<T, P, 4, 4>(a, grid, stream);
        else backward_types<T, P, 4, 2>(a, grid, stream);
    } else {
        if (h4) backward_types<T, P, 2, 4>(a, grid, stream);
        else backward_types<T, P, 2, 2>(a, grid, stream);
    }
}

}  // namespace

int32_t norm_backward_parts(int64_t rows, int32_t cols) {
    (void)cols;
    return static_cast<int32_t>(rows < ZERO_NORM_MAX_PARTS ? rows : ZERO_NORM_MAX_PARTS);
}

hipError_t launch_rmsnorm_backward(const NormBackwardArgs& a, hipStream_t stream) {
    const int c = a.cols;
    const int parts = norm_backward_parts(a.rows, c);
    if (parts > 0) {
        const dim3 grid(static_cast<uint32_t>(parts));
        if (c <= 512) backward_shape<64, 1>(a, grid, stream);
        else if (c <= 1024) backward_shape<64, 2>(a, grid, stream);
        else if (c <= 2048) backward_shape<128, 2>(a, grid, stream);
        else if (c <= 4096) backward_shape<256, 2>(a, grid, stream);
        else if (c <= 8192) backward_shape<512, 2>(a, grid, stream);
        else if (c <= 16384) backward_shape<1024, 2>(a, grid, stream);
        else if (c <= 32768) backward_shape<1024, 4>(a, grid, stream);
        else backward_shape<1024, 8>(a, grid, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.dw) {
        const dim3 grid(static_cast<uint32_t>((c + kDwCols - 1) / kDwCols));
        rmsnorm_dw_kernel<<<grid, kDwCols * kDwGroups, 0, stream>>>(a.parts, parts, c, a.dw,
                                                                    a.dw_dtype);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace zero
