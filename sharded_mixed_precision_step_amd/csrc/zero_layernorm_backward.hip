// Gradients of the layer norm.
//
// dx needs two sums over its row, mean(g) and mean(g xhat); dw and db are sums over
// rows.  Bound by HBM: one pass over the arrays for rows of 8 to 16,384 columns.
// 16387 x 1001 bf16 with dresidual: 26 us for dx and the partial rows (5.1 TB/s), 4.7 for
// dw and db from them; 8192 x 4096 fp16 56 us, 59 to 63 with dresidual.
#include "zero_device.h"
#include "zero_model_internal.h"

namespace zero {
namespace {

using namespace dev;

__device__ __forceinline__ void load_elements(const void* p, int64_t i, int n, int dtype,
                                              float (&f)[8]) {
    if (dtype == ZERO_F32) widen8<4>(load8<4>(p, i, n), false, f);
    else widen8<2>(load8<2>(p, i, n), dtype == ZERO_BF16, f);
}

// ---- rows in registers -----------------------------------------------------

// Eight columns of one row, as loaded.
template <int DB, int HB, int RB>
struct Pack {
    Raw8<DB> d;
    Raw8<HB> h;
    Raw8<RB == 0 ? 2 : RB> r;
    __device__ __forceinline__ void load(const LayerNormBackwardArgs& a, int64_t row, int c) {
        d = load8<DB>(a.dy, row * a.ld_dy + c, 8);
        h = load8<HB>(a.h, row * a.ld_h + c, 8);
        if constexpr (RB != 0) r = load8<RB>(a.dres, row * a.ld_dr + c, 8);
    }
    // Sums of g and g xhat, of the elements from `from` on.  Behind it all loads have
    // arrived: dx may be any of the three, and its owner's pack may share elements with
    // the row's last one.
    __device__ __forceinline__ void reduce(const LayerNormBackwardArgs& a, const float (&w)[8],
                                           int from, float mean, float rstd, float& sg,
                                           float& sgx) const {
        float dy[8], x[8];
        widen8<DB>(d, a.dy_dtype == ZERO_BF16, dy);
        widen8<HB>(h, a.h_dtype == ZERO_BF16, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float g = k >= from ? dy[k] * w[k] : 0.0f;
            sg += g;
            sgx = __builtin_fmaf(g, k >= from ? (x[k] - mean) * rstd : 0.0f, sgx);
        }
        if constexpr (RB != 0) arrived(r);
    }
    __device__ __forceinline__ void finish(const LayerNormBackwardArgs& a, int64_t row, int c,
                                           const float (&w)[8], float mean, float rstd, float mg,
                                           float mgx, float (&dw)[8], float (&db)[8]) const {
        float dy[8], x[8], dr[8] = {};
        widen8<DB>(d, a.dy_dtype == ZERO_BF16, dy);
        widen8<HB>(h, a.h_dtype == ZERO_BF16, x);
        if constexpr (RB != 0) widen8<RB>(r, a.dr_dtype == ZERO_BF16, dr);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float xhat = (x[k] - mean) * rstd;
            dw[k] = __builtin_fmaf(dy[k], xhat, dw[k]);
            db[k] += dy[k];
            const float inner = __builtin_fmaf(-xhat, mgx, dy[k] * w[k] - mg);
            dy[k] = __builtin_fmaf(rstd, inner, dr[k]);
        }
        store8(a.dx, row * a.ld_dx + c, 8, a.dx_dtype, dy);
    }
};

// Sums of x and y over a row's lanes: LPR neighbouring lanes of a wave (16, 32 or
// 64), or the workgroup (LPR 0), with one barrier.  `part` holds two floats a wave,
// and two calls may not share it without a barrier between them.
template <int LPR>
__device__ __forceinline__ void row_sums(float& x, float& y, float (*part)[2]) {
    constexpr int kLanes = LPR == 0 ? 64 : LPR;
#pragma unroll
    for (int d = 1; d < kLanes; d *= 2) {
        x += __shfl_xor(x, d);
        y += __shfl_xor(y, d);
    }
    if constexpr (LPR == 0) {
        const int waves = static_cast<int>(blockDim.x >> 6);
        if ((threadIdx.x & 63) == 0) {
            part[threadIdx.x >> 6][0] = x;
            part[threadIdx.x >> 6][1] = y;
        }
        __syncthreads();
        x = part[0][0];
        y = part[0][1];
        for (int w = 1; w < waves; ++w) {
            x += part[w][0];
            y += part[w][1];
        }
    }
}

// A row's lanes (LPR of a wave, or the workgroup) take one row after another and keep
// the same columns, so that the sums for dw and db over those rows stay in registers;
// the workgroup's leave once, as one fp32 partial row each.  The next row's loads are
// under way during this one's sums where registers allow it (one pack a lane, or two
// of 16-bit types in a wave).
//
// Where a row's length is no multiple of eight, its last pack is its last eight
// elements: what it shares with the pack before goes into the row's sums once, and
// comes out of both alike.  (A tail loaded by elements stops its wave.)
template <int MAX_T, int LPR, int P, int DB, int HB, int RB>
__global__ __launch_bounds__(MAX_T) void layernorm_backward_kernel(const LayerNormBackwardArgs a) {
    constexpr bool kAhead = P == 1 || (LPR != 0 && DB == 2 && HB == 2);
    constexpr int kGroups = LPR == 0 ? 1 : MAX_T / LPR;
    __shared__ float part[2][16][2];
    // columns' sums of each group of lanes, dw and db in turn
    __shared__ float sums[LPR == 0 ? 1 : kGroups][LPR == 0 ? 1 : LPR * P * 8];
    const int T = LPR == 0 ? static_cast<int>(blockDim.x) : LPR;
    const int lane = LPR == 0 ? static_cast<int>(threadIdx.x) : threadIdx.x % LPR;
    const int group = LPR == 0 ? 0 : threadIdx.x / LPR;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    // where pack i of the lane starts, and how many of its elements are another's
    int at[P], from[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * T + lane) * 8;
        at[i] = c > a.cols - 8 ? a.cols - 8 : c;
        from[i] = c - at[i];
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kGroups + group;
    float dw[P][8] = {}, db[P][8] = {}, w[P][8];
    Pack<DB, HB, RB> next[kAhead ? P : 1];
    float next_mean = 0.0f, next_rstd = 0.0f;
    if constexpr (kAhead) {
        if (row0 < a.rows) {
            next_mean = a.mean[row0];
            next_rstd = a.rstd[row0];
#pragma unroll
            for (int i = 0; i < P; ++i) next[i].load(a, row0, at[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) load_elements(a.weight, at[i], 8, a.w_dtype, w[i]);
    int flip = 0;
    for (int64_t row = row0; row < a.rows; row += step, flip ^= 1) {
        Pack<DB, HB, RB> now[P];
        float mean, rstd;
        if constexpr (kAhead) {
            mean = next_mean;
            rstd = next_rstd;
#pragma unroll
            for (int i = 0; i < P; ++i) now[i] = next[i];
            if (row + step < a.rows) {
                next_mean = a.mean[row + step];
                next_rstd = a.rstd[row + step];
#pragma unroll
                for (int i = 0; i < P; ++i) next[i].load(a, row + step, at[i]);
            }
        } else {
            mean = a.mean[row];
            rstd = a.rstd[row];
#pragma unroll
            for (int i = 0; i < P; ++i) now[i].load(a, row, at[i]);
        }
        float sg = 0.0f, sgx = 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) now[i].reduce(a, w[i], from[i], mean, rstd, sg, sgx);
        row_sums<LPR>(sg, sgx, part[flip]);
        const float mg = sg * inv_cols, mgx = sgx * inv_cols;
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (from[i] < 8)
                now[i].finish(a, row, at[i], w[i], mean, rstd, mg, mgx, dw[i], db[i]);
    }
    if (!a.parts) return;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float(&v)[P][8] = which ? db : dw;
        const int64_t out = (which * static_cast<int64_t>(gridDim.x) + blockIdx.x) * a.cols;
        if constexpr (LPR == 0) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (from[i] < 8) store8(a.parts, out + at[i], 8, ZERO_F32, v[i]);
        } else {
            if (which) __syncthreads();
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (from[i] >= 8) continue;
#pragma unroll
                for (int k = 0; k < 8; ++k) sums[group][at[i] + k] = v[i][k];
            }
            __syncthreads();
            for (int c = threadIdx.x; c < a.cols; c += MAX_T) {
                float s = sums[0][c];
#pragma unroll
                for (int g = 1; g < kGroups; ++g) s += sums[g][c];
                a.parts[out + c] = s;
            }
        }
    }
}

// ---- rows read twice -------------------------------------------------------
// Wider rows have more sums for dw and db than a lane's registers hold, and rows of
// less than 8 columns no eight elements: dw and db by columns first, then dx by rows.

constexpr int kLanes = 256;

__global__ __launch_bounds__(kLanes) void layernorm_dx_kernel(const LayerNormBackwardArgs a,
                                                              int64_t first) {
    __shared__ float part[kLanes / 64][2];
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
    row_sums<0>(sg, sgx, part);
    const float mg = sg * inv_cols, mgx = sgx * inv_cols;
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

// ---- dw and db from the partial rows ---------------------------------------

// dw (blockIdx.y == 0) and db: 64 columns per workgroup, 16 groups of lanes over the
// partial rows, then over the groups, in a fixed order.  Up to 2,048 columns 32 and
// 32, so that there are workgroups enough.
constexpr int kDwThreads = 1024;
template <int kDwCols>
__global__ __launch_bounds__(kDwThreads) void layernorm_dw_kernel(const float* parts, int n_parts,
                                                                  int cols, void* dw, void* db,
                                                                  int dtype) {
    constexpr int kDwGroups = kDwThreads / kDwCols;
    __shared__ float sums[kDwGroups][kDwCols];
    void* out = blockIdx.y ? db : dw;
    if (!out) return;
    parts += blockIdx.y * static_cast<int64_t>(n_parts) * cols;
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
        store1(out, c, dtype, v);
    }
}

// How a row's width is dealt with: lanes of a wave per row, or 0 for the workgroup,
// or -1 for rows read twice.  (16387 x 1001 bf16: 150 us read twice, 30 by a wave; 1024 x
// 32768 fp16, read twice, 100 us, 2.0 TB/s, 127 with dresidual.)
int lanes_per_row(int cols) {
    if (cols < 8 || cols > 16384) return -1;
    return cols <= 128 ? 16 : cols <= 256 ? 32 : cols <= 1024 ? 64 : 0;
}
constexpr int kNarrowLanes = 256;  // of a workgroup with several rows

template <int MAX_T, int LPR, int P>
hipError_t held(const LayerNormBackwardArgs& a, uint32_t grid, hipStream_t stream) {
    const uint32_t block = LPR != 0 ? MAX_T
                                    : static_cast<uint32_t>((a.cols + P * 512 - 1) / (P * 512) * 64);
    const bool d4 = a.dy_dtype == ZERO_F32, h4 = a.h_dtype == ZERO_F32;
    const int rb = !a.dres ? 0 : a.dr_dtype == ZERO_F32 ? 4 : 2;
    auto run = [&](auto kernel) {
        kernel<<<grid, block, 0, stream>>>(a);
        return hipGetLastError();
    };
#define ZERO_LN_RES(D, H)                                                  \
    (rb == 0   ? run(layernorm_backward_kernel<MAX_T, LPR, P, D, H, 0>)    \
     : rb == 4 ? run(layernorm_backward_kernel<MAX_T, LPR, P, D, H, 4>)    \
               : run(layernorm_backward_kernel<MAX_T, LPR, P, D, H, 2>))
    if (d4) return h4 ? ZERO_LN_RES(4, 4) : ZERO_LN_RES(4, 2);
    return h4 ? ZERO_LN_RES(2, 4) : ZERO_LN_RES(2, 2);
#undef ZERO_LN_RES
}

}  // namespace

// Workgroups, each with a partial row of dw and one of db: two a CU where the rows are
// many and the partial rows short, else one, since what dw's kernel adds up grows with them.
int32_t layernorm_backward_parts(int64_t rows, int32_t cols) {
    const int lpr = lanes_per_row(cols);
    const int64_t groups = lpr > 0 ? kNarrowLanes / lpr : 1;
    int64_t parts = lpr > 0 ? 512 : cols <= 2048 ? 512 : 256;
    while (parts > 256 && rows < 4 * parts * groups) parts /= 2;
    const int64_t most = (rows + groups - 1) / groups;
    return static_cast<int32_t>(most < parts ? most : parts);
}

hipError_t launch_layernorm_backward(const LayerNormBackwardArgs& a, hipStream_t stream) {
    const int c = a.cols, lpr = lanes_per_row(c);
    const int parts = layernorm_backward_parts(a.rows, c);
    if (parts > 0) {
        const uint32_t grid = static_cast<uint32_t>(parts);
        hipError_t e = hipSuccess;
        if (lpr == 16) e = held<kNarrowLanes, 16, 1>(a, grid, stream);
        else if (lpr == 32) e = held<kNarrowLanes, 32, 1>(a, grid, stream);
        else if (lpr == 64 && c <= 512) e = held<kNarrowLanes, 64, 1>(a, grid, stream);
        else if (lpr == 64) e = held<kNarrowLanes, 64, 2>(a, grid, stream);
        else if (lpr == 0 && c <= 8192) e = held<1024, 0, 1>(a, grid, stream);
        else if (lpr == 0) e = held<1024, 0, 2>(a, grid, stream);
        else {
            if (a.parts) {  // before dx, which may take the place of dy or h
                const dim3 by(static_cast<uint32_t>((c + 8 * kLanes - 1) / (8 * kLanes)), grid);
                layernorm_parts_kernel<<<by, kLanes, 0, stream>>>(a);
                e = hipGetLastError();
            }
            if (e == hipSuccess)
                e = in_launches(a.rows, kLanes, [&](int64_t first, uint32_t n) {
                    layernorm_dx_kernel<<<n, kLanes, 0, stream>>>(a, first);
                    return hipGetLastError();
                });
        }
        if (e != hipSuccess) return e;
    }
    if (a.dw || a.db) {
        auto run = [&](auto kernel, int per) {
            kernel<<<dim3(static_cast<uint32_t>((c + per - 1) / per), 2), kDwThreads, 0, stream>>>(
                a.parts, parts, c, a.dw, a.db, a.dw_dtype);
        };
        if (c <= 2048) run(layernorm_dw_kernel<32>, 32);
        else run(layernorm_dw_kernel<64>, 64);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace zero
