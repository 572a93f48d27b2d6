// Gradients of the layer norm.
//
// dx needs two sums over its row, mean(g) and mean(g xhat); dw and db are sums
// over rows.  Bound by HBM.
#include "zero_device.h"
#include "zero_model_internal.h"

namespace zero {
namespace {

using namespace dev;

constexpr int kLanes = 256;

__device__ __forceinline__ void load_elements(const void* p, int64_t i, int n, int dtype,
                                              float (&f)[8]) {
    if (dtype == ZERO_F32) widen8<4>(load8<4>(p, i, n), false, f);
    else widen8<2>(load8<2>(p, i, n), dtype == ZERO_BF16, f);
}

// One workgroup per row, which it reads twice.
__global__ __launch_bounds__(kLanes) void layernorm_dx_kernel(const LayerNormBackwardArgs a,
                                                              int64_t first) {
    __shared__ float part[2][16];
    const int64_t row = first + blockIdx.x;
    const float mean = a.mean[row], rstd = a.rstd[row];
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    float sg = 0.0f, sgx = 0.0f;
    for (int c = threadIdx.x * 8; c < a.cols; c += kLanes * 8) {
        float dy[8], h[8], w[8];
        load_elements(a.dy, row * a.ld_dy + c, a.cols - c, a.dy_dtype, dy);
        load_elements(a.h, row * a.ld_h + c, a.cols - c, a.h_dtype, h);
        load_elements(a.weight, c, a.cols - c, a.w_dtype, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float g = dy[k] * w[k];
            sg += g;
            const float sum = __builtin_fmaf(g, (h[k] - mean) * rstd, sgx);
            sgx = c + k < a.cols ? sum : sgx;
        }
    }
    const float mg = block_sum(sg, part[0]) * inv_cols;
    const float mgx = block_sum(sgx, part[1]) * inv_cols;
    for (int c = threadIdx.x * 8; c < a.cols; c += kLanes * 8) {
        float dy[8], h[8], w[8], dr[8] = {};
        load_elements(a.dy, row * a.ld_dy + c, a.cols - c, a.dy_dtype, dy);
        load_elements(a.h, row * a.ld_h + c, a.cols - c, a.h_dtype, h);
        load_elements(a.weight, c, a.cols - c, a.w_dtype, w);
        if (a.dres) load_elements(a.dres, row * a.ld_dr + c, a.cols - c, a.dr_dtype, dr);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float xhat = (h[k] - mean) * rstd;
            const float inner = __builtin_fmaf(-xhat, mgx, dy[k] * w[k] - mg);
            dy[k] = __builtin_fmaf(rstd, inner, dr[k]);
        }
        store8(a.dx, row * a.ld_dx + c, a.cols - c, a.dx_dtype, dy);
    }
}

// 2,048 columns of the rows blockIdx.y, + gridDim.y, ..: partial rows of dw, db.
__global__ __launch_bounds__(kLanes) void layernorm_parts_kernel(const LayerNormBackwardArgs a) {
    const int c = static_cast<int>(blockIdx.x * kLanes + threadIdx.x) * 8;
    if (c >= a.cols) return;
    float dw[8] = {}, db[8] = {};
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float mean = a.mean[row], rstd = a.rstd[row];
        float dy[8], h[8];
        load_elements(a.dy, row * a.ld_dy + c, a.cols - c, a.dy_dtype, dy);
        load_elements(a.h, row * a.ld_h + c, a.cols - c, a.h_dtype, h);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            dw[k] = __builtin_fmaf(dy[k], (h[k] - mean) * rstd, dw[k]);
            db[k] += dy[k];
        }
    }
    const int64_t half = static_cast<int64_t>(gridDim.y) * a.cols;
    store8(a.parts, blockIdx.y * static_cast<int64_t>(a.cols) + c, a.cols - c, ZERO_F32, dw);
    store8(a.parts, half + blockIdx.y * static_cast<int64_t>(a.cols) + c, a.cols - c, ZERO_F32, db);
}

// dw (blockIdx.y == 0) and db = the partial rows' sum: 64 columns per workgroup,
// 16 groups of lanes over the partial rows, then over the groups.
constexpr int kDwThreads = 1024, kDwCols = 64, kDwGroups = kDwThreads / kDwCols;
__global__ __launch_bounds__(kDwThreads) void layernorm_dw_kernel(const float* parts, int n_parts,
                                                                  int cols, void* dw, void* db,
                                                                  int dtype) {
    __shared__ float sums[kDwGroups][kDwCols];
    void* out = blockIdx.y ? db : dw;
    if (!out) return;
    parts += blockIdx.y * static_cast<int64_t>(n_parts) * cols;
    const int lane = threadIdx.x % kDwCols, group = threadIdx.x / kDwCols;
    const int c = blockIdx.x * kDwCols + lane;
    float v = 0.0f;
    if (c < cols)
        for (int p = group; p < n_parts; p += kDwGroups)
            v += parts[static_cast<int64_t>(p) * cols + c];
    sums[group][lane] = v;
    __syncthreads();
    if (group == 0 && c < cols) {
        for (int g = 1; g < kDwGroups; ++g) v += sums[g][lane];
        store1(out, c, dtype, v);
    }
}

}  // namespace

int32_t layernorm_backward_parts(int64_t rows, int32_t) {
    return static_cast<int32_t>(rows < 256 ? rows : 256);
}

hipError_t launch_layernorm_backward(const LayerNormBackwardArgs& a, hipStream_t stream) {
    const int parts = layernorm_backward_parts(a.rows, a.cols);
    if (a.parts && parts > 0) {  // before dx, which may take the place of dy or h
        const dim3 grid(static_cast<uint32_t>((a.cols + 8 * kLanes - 1) / (8 * kLanes)),
                        static_cast<uint32_t>(parts));
        layernorm_parts_kernel<<<grid, kLanes, 0, stream>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.rows > 0) {
        const hipError_t e = in_launches(a.rows, kLanes, [&](int64_t first, uint32_t grid) {
            layernorm_dx_kernel<<<grid, kLanes, 0, stream>>>(a, first);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    }
    if (a.dw || a.db) {
        const dim3 grid(static_cast<uint32_t>((a.cols + kDwCols - 1) / kDwCols), 2);
        layernorm_dw_kernel<<<grid, kDwThreads, 0, stream>>>(a.parts, parts, a.cols, a.dw, a.db,
                                                             a.dw_dtype);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace zero
