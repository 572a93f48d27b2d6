// Gradients of the root-mean-square norm.
//
// One pass over its arrays, bound by HBM, with the forward's row layout (one
// workgroup per row, eight elements per lane and step).
#include "zero_device.h"
#include "zero_train_internal.h"

namespace zero {
namespace {

using namespace dev;

// Eight columns of one row, as loaded.
template <int DB, int HB, int RB>
struct Pack {
    Raw8<DB> d;
    Raw8<HB> h;
    Raw8<RB == 0 ? 2 : RB> r;
    __device__ __forceinline__ void load(const NormBackwardArgs& a, int64_t row, int c) {
        d = load8<DB>(a.dy, row * a.ld_dy + c, a.cols - c);
        h = load8<HB>(a.h, row * a.ld_h + c, a.cols - c);
        if constexpr (RB != 0) r = load8<RB>(a.dres, row * a.ld_dr + c, a.cols - c);
    }
    // dot += g . xhat
    __device__ __forceinline__ void reduce(const NormBackwardArgs& a, const float (&w)[8],
                                           float rstd, float& dot) const {
        float dy[8], x[8];
        widen8<DB>(d, a.dy_dtype == ZERO_BF16, dy);
        widen8<HB>(h, a.h_dtype == ZERO_BF16, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) dot = __builtin_fmaf(dy[k] * w[k], x[k] * rstd, dot);
    }
    __device__ __forceinline__ void finish(const NormBackwardArgs& a, int64_t row, int c,
                                           const float (&w)[8], float rstd, float mean,
                                           float (&dw)[8]) const {
        float dy[8], x[8], dr[8];
        widen8<DB>(d, a.dy_dtype == ZERO_BF16, dy);
        widen8<HB>(h, a.h_dtype == ZERO_BF16, x);
        if constexpr (RB != 0) widen8<RB>(r, a.dr_dtype == ZERO_BF16, dr);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float xhat = x[k] * rstd;
            dw[k] = __builtin_fmaf(dy[k], xhat, dw[k]);
            const float inner = __builtin_fmaf(-xhat, mean, dy[k] * w[k]);
            if constexpr (RB != 0) dy[k] = __builtin_fmaf(rstd, inner, dr[k]);
            else dy[k] = rstd * inner;
        }
        store8(a.dx, row * a.ld_dx + c, a.cols - c, a.dx_dtype, dy);
    }
};

__device__ __forceinline__ void load_weight(const NormBackwardArgs& a, int c, float (&w)[8]) {
    if (a.w_dtype == ZERO_F32) widen8<4>(load8<4>(a.weight, c, a.cols - c), false, w);
    else widen8<2>(load8<2>(a.weight, c, a.cols - c), a.w_dtype == ZERO_BF16, w);
}

// A workgroup takes rows blockIdx.x, + gridDim.x, ...  Its lanes keep the same
// columns for every row, so dw's sum over those rows stays in registers and
// leaves once, as one fp32 partial row.  Up to 16,384 columns a row is held in
// registers, and up to 8,192 the next one's loads are under way meanwhile (one
// pack per lane: more waves for the arithmetic of the one row, 1003 x 5001 17 us
// against 20 with two packs); wider rows are read again behind the reduction.
template <int MAX_T, int P, int DB, int HB, int RB>
__global__ __launch_bounds__(MAX_T) void rmsnorm_backward_kernel(const NormBackwardArgs a) {
    __shared__ float part[2][16];
    constexpr bool kHeld = P <= 2, kAhead = P == 1;
    const int T = static_cast<int>(blockDim.x);
    const int first = static_cast<int>(threadIdx.x) * 8;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    float dw[P][8] = {}, w[kHeld ? P : 1][8];
    Pack<DB, HB, RB> next[kAhead ? P : 1];
    float next_rstd = 0.0f;
    if constexpr (kAhead) {
        next_rstd = a.rstd[blockIdx.x];
#pragma unroll
        for (int i = 0; i < P; ++i) next[i].load(a, blockIdx.x, first + i * T * 8);
    }
    if constexpr (kHeld) {
#pragma unroll
        for (int i = 0; i < P; ++i) load_weight(a, first + i * T * 8, w[i]);
    }
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
        float dot = 0.0f;
        if constexpr (kHeld) {
            Pack<DB, HB, RB> now[P];
            float rstd;
            if constexpr (kAhead) {
                rstd = next_rstd;
#pragma unroll
                for (int i = 0; i < P; ++i) now[i] = next[i];
                if (row + gridDim.x < a.rows) {
                    next_rstd = a.rstd[row + gridDim.x];
#pragma unroll
                    for (int i = 0; i < P; ++i) next[i].load(a, row + gridDim.x, first + i * T * 8);
                }
            } else {
                rstd = a.rstd[row];
#pragma unroll
                for (int i = 0; i < P; ++i) now[i].load(a, row, first + i * T * 8);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) now[i].reduce(a, w[i], rstd, dot);
            const float mean = block_sum(dot, part[flip]) * inv_cols;
#pragma unroll
            for (int i = 0; i < P; ++i)
                now[i].finish(a, row, first + i * T * 8, w[i], rstd, mean, dw[i]);
        } else {
            const float rstd = a.rstd[row];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                Pack<DB, HB, RB> now;
                now.load(a, row, first + i * T * 8);
                load_weight(a, first + i * T * 8, w[0]);
                now.reduce(a, w[0], rstd, dot);
            }
            const float mean = block_sum(dot, part[flip]) * inv_cols;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                Pack<DB, HB, RB> now;
                now.load(a, row, first + i * T * 8);
                load_weight(a, first + i * T * 8, w[0]);
                now.finish(a, row, first + i * T * 8, w[0], rstd, mean, dw[i]);
                __builtin_amdgcn_sched_barrier(0);  // one pack's registers at a time
            }
        }
    }
    if (!a.parts) return;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = first + i * T * 8;
        store8(a.parts, static_cast<int64_t>(blockIdx.x) * a.cols + c, a.cols - c, ZERO_F32,
               dw[i]);
    }
}

// dw = the partial rows' sum: 64 columns per workgroup, 16 groups of lanes
// over the partial rows, then over the groups, in a fixed order.
constexpr int kDwCols = 64;
constexpr int kDwGroups = 16;
__global__ __launch_bounds__(kDwCols * kDwGroups) void rmsnorm_dw_kernel(const float* parts,
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

template <int MAX_T, int P, int DB, int HB>
void backward_types(const NormBackwardArgs& a, dim3 grid, dim3 block, hipStream_t stream) {
    if (!a.dres) rmsnorm_backward_kernel<MAX_T, P, DB, HB, 0><<<grid, block, 0, stream>>>(a);
    else if (a.dr_dtype == ZERO_F32)
        rmsnorm_backward_kernel<MAX_T, P, DB, HB, 4><<<grid, block, 0, stream>>>(a);
    else rmsnorm_backward_kernel<MAX_T, P, DB, HB, 2><<<grid, block, 0, stream>>>(a);
}

template <int MAX_T, int P>
void backward_shape(const NormBackwardArgs& a, dim3 grid, hipStream_t stream) {
    const dim3 block(static_cast<uint32_t>((a.cols + P * 512 - 1) / (P * 512) * 64));
    const bool d4 = a.dy_dtype == ZERO_F32, h4 = a.h_dtype == ZERO_F32;
    if (d4) {
        if (h4) backward_types<MAX_T, P, 4, 4>(a, grid, block, stream);
        else backward_types<MAX_T, P, 4, 2>(a, grid, block, stream);
    } else {
        if (h4) backward_types<MAX_T, P, 2, 4>(a, grid, block, stream);
        else backward_types<MAX_T, P, 2, 2>(a, grid, block, stream);
    }
}

}  // namespace

// One workgroup per CU: beyond that dw's partial rows cost more than the extra
// rows in flight bring.  8192 x 4096 (fp16 dy and dx, fp32 h): 65.7 us with 256,
// 5.1 TB/s, 69.2 with 512; 1003 x 5001 in bf16: 19.7 and 21.8, of which 5 are its
// rows' odd addresses.
int32_t norm_backward_parts(int64_t rows, int32_t cols) {
    (void)cols;
    constexpr int64_t kMost = 256;
    static_assert(kMost <= ZERO_NORM_MAX_PARTS, "the documented limit");
    return static_cast<int32_t>(rows < kMost ? rows : kMost);
}

hipError_t launch_rmsnorm_backward(const NormBackwardArgs& a, hipStream_t stream) {
    const int c = a.cols;
    const int parts = norm_backward_parts(a.rows, c);
    if (parts > 0) {
        const dim3 grid(static_cast<uint32_t>(parts));
        if (c <= 512) backward_shape<64, 1>(a, grid, stream);
        else if (c <= 8192) backward_shape<1024, 1>(a, grid, stream);
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
