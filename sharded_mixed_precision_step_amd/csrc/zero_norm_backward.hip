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
    __device__ __forceinline__ void load(const NormBackwardArgs& a, int64_t row, int c, int n) {
        d = load8<DB>(a.dy, row * a.ld_dy + c, n);
        h = load8<HB>(a.h, row * a.ld_h + c, n);
        if constexpr (RB != 0) r = load8<RB>(a.dres, row * a.ld_dr + c, n);
    }
    // dot += g . xhat, of the elements from `from` on
    __device__ __forceinline__ void reduce(const NormBackwardArgs& a, const float (&w)[8], int from,
                                           float rstd, float& dot) const {
        float dy[8], x[8];
        widen8<DB>(d, a.dy_dtype == ZERO_BF16, dy);
        widen8<HB>(h, a.h_dtype == ZERO_BF16, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float sum = __builtin_fmaf(dy[k] * w[k], x[k] * rstd, dot);
            dot = k >= from ? sum : dot;
        }
        // dx may be dresidual, and a held row's last pack shares another lane's elements
        if constexpr (RB != 0) arrived(r);
    }
    __device__ __forceinline__ void finish(const NormBackwardArgs& a, int64_t row, int c, int n,
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
        store8(a.dx, row * a.ld_dx + c, n, a.dx_dtype, dy);
    }
};

__device__ __forceinline__ void load_weight(const NormBackwardArgs& a, int c, int n,
                                            float (&w)[8]) {
    if (a.w_dtype == ZERO_F32) widen8<4>(load8<4>(a.weight, c, n), false, w);
    else widen8<2>(load8<2>(a.weight, c, n), a.w_dtype == ZERO_BF16, w);
}

// A workgroup takes rows blockIdx.x, + gridDim.x, ...  Its lanes keep the same
// columns for every row, so dw's sum over those rows stays in registers and
// leaves once, as one fp32 partial row.  Up to 16,384 columns a row is held in
// registers, and up to 8,192 the next one's loads are under way meanwhile (one
// pack per lane: more waves for the arithmetic of the one row, 1003 x 5001 17 us
// against 20 with two packs); wider rows are read again behind the reduction.
// Those (and rows of less than 8 columns) also have more sums for dw and packs than
// a lane's 128 registers hold, and spill: fp16, 1024 x 32768 132 us, 1.5 TB/s, 1024
// x 65536 599.  Narrow rows leave lanes without elements, one wave to a row: 262144
// x 128 201 us, 1.0 TB/s; 65536 x 256 56 us, 1.8.
//
// Where a row's length is no multiple of eight, a held row's last pack is its
// last eight elements: what it shares with the pack before goes into the row's
// sum once, and comes out of both alike.  (A tail loaded by elements stops its
// wave until they are there, and the next row's loads with it: 8000 x 5001 in
// bf16 117 us, 8000 x 5000 60.)  Rows read twice may not, since dx may be dy.
template <int MAX_T, int P, int DB, int HB, int RB>
__global__ __launch_bounds__(MAX_T) void rmsnorm_backward_kernel(const NormBackwardArgs a) {
    __shared__ float part[2][16];
    constexpr bool kHeld = P <= 2, kAhead = P == 1;
    const int T = static_cast<int>(blockDim.x);
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    // where pack i of the lane starts, its elements, and how many are another's
    int at[P], n[P], from[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * T + static_cast<int>(threadIdx.x)) * 8;
        at[i] = kHeld && c > a.cols - 8 ? a.cols - 8 : c;
        n[i] = kHeld ? 8 : a.cols - c;
        from[i] = c - at[i];
    }
    float dw[P][8] = {}, w[kHeld ? P : 1][8];
    Pack<DB, HB, RB> next[kAhead ? P : 1];
    float next_rstd = 0.0f;
    if constexpr (kAhead) {
        next_rstd = a.rstd[blockIdx.x];
#pragma unroll
        for (int i = 0; i < P; ++i) next[i].load(a, blockIdx.x, at[i], n[i]);
    }
    if constexpr (kHeld) {
#pragma unroll
        for (int i = 0; i < P; ++i) load_weight(a, at[i], n[i], w[i]);
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
                    for (int i = 0; i < P; ++i) next[i].load(a, row + gridDim.x, at[i], n[i]);
                }
            } else {
                rstd = a.rstd[row];
#pragma unroll
                for (int i = 0; i < P; ++i) now[i].load(a, row, at[i], n[i]);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) now[i].reduce(a, w[i], from[i], rstd, dot);
            const float mean = block_sum(dot, part[flip]) * inv_cols;
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (from[i] < 8) now[i].finish(a, row, at[i], n[i], w[i], rstd, mean, dw[i]);
        } else {
            const float rstd = a.rstd[row];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                Pack<DB, HB, RB> now;
                now.load(a, row, at[i], n[i]);
                load_weight(a, at[i], n[i], w[0]);
                now.reduce(a, w[0], 0, rstd, dot);
            }
            const float mean = block_sum(dot, part[flip]) * inv_cols;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                Pack<DB, HB, RB> now;
                now.load(a, row, at[i], n[i]);
                load_weight(a, at[i], n[i], w[0]);
                now.finish(a, row, at[i], n[i], w[0], rstd, mean, dw[i]);
                __builtin_amdgcn_sched_barrier(0);  // one pack's registers at a time
            }
        }
    }
    if (!a.parts) return;
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (from[i] < 8)
            store8(a.parts, static_cast<int64_t>(blockIdx.x) * a.cols + at[i], n[i], ZERO_F32,
                   dw[i]);
}

// dw = the partial rows' sum: 64 columns per workgroup, 16 groups of lanes
// over the partial rows, then over the groups, in a fixed order.  Up to 2,048
// columns 32 and 32, so that there are workgroups enough (8192 x 1024, 1,024
// partial rows: 4.8 us, 6.0 with 64 and 16; 5,001 columns, 256 rows: 4.9 and 4.4).
constexpr int kDwThreads = 1024;
template <int kDwCols>
__global__ __launch_bounds__(kDwThreads) void rmsnorm_dw_kernel(const float* parts, int n_parts,
                                                                int cols, void* dw, int dtype) {
    constexpr int kDwGroups = kDwThreads / kDwCols;
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

// Workgroups, each with a partial row of dw.  One per CU beyond 2,048 columns:
// more rows at a time bring less than their partial rows cost (8192 x 4096, fp16
// dy and dx, fp32 h: 65 us with 256, 5.1 TB/s, 69 with 512).  Narrower rows are
// few waves each and need more of them to fill the CUs, four rows each at least
// (bf16, 8192 x 1024: 20 us with 1,024, 36 with 256; 1003 x 1024: 9 with 256, 12
// with 1,003).
//
// 1003 x 5001 in bf16: 15.1 us, of which the sum of the partial rows is 4.4; rows
// at odd addresses cost little there, a fifth at 8000 rows (80 us, 70).
int32_t norm_backward_parts(int64_t rows, int32_t cols) {
    int64_t parts = cols <= 1024 ? 1024 : cols <= 2048 ? 512 : 256;
    static_assert(ZERO_NORM_MAX_PARTS >= 1024, "the documented limit");
    while (parts > 256 && rows < 4 * parts) parts /= 2;
    return static_cast<int32_t>(rows < parts ? rows : parts);
}

hipError_t launch_rmsnorm_backward(const NormBackwardArgs& a, hipStream_t stream) {
    const int c = a.cols;
    const int parts = norm_backward_parts(a.rows, c);
    if (parts > 0) {
        const dim3 grid(static_cast<uint32_t>(parts));
        if (c < 8) backward_shape<1024, 4>(a, grid, stream);  // no eight elements: by elements
        else if (c <= 512) backward_shape<64, 1>(a, grid, stream);
        else if (c <= 8192) backward_shape<1024, 1>(a, grid, stream);
        else if (c <= 16384) backward_shape<1024, 2>(a, grid, stream);
        else if (c <= 32768) backward_shape<1024, 4>(a, grid, stream);
        else backward_shape<1024, 8>(a, grid, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.dw) {
        auto run = [&](auto kernel, int per) {
            kernel<<<static_cast<uint32_t>((c + per - 1) / per), kDwThreads, 0, stream>>>(
                a.parts, parts, c, a.dw, a.dw_dtype);
        };
        if (c <= 2048) run(rmsnorm_dw_kernel<32>, 32);
        else run(rmsnorm_dw_kernel<64>, 64);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace zero
