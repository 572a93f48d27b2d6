// Residual addition and layer norm.
//
// One pass over its arrays, bound by HBM: a row's elements stay in registers as
// fp32, between the sum for the mean, the sum of squares about that mean (two
// reductions, so that a row far from zero keeps its variance) and the outputs.
#include "zero_device.h"
#include "zero_model_internal.h"

namespace zero {
namespace {

using namespace dev;

template <int MAX_T, int P, int XB, int RB>
__global__ __launch_bounds__(MAX_T) void layernorm_kernel(const LayerNormArgs a, int64_t first) {
    __shared__ float part[2][16];
    const int T = static_cast<int>(blockDim.x);
    const int64_t row = first + blockIdx.x;
    const int t = threadIdx.x;
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    Raw8<XB> rx[P];
    Raw8<RB == 0 ? 2 : RB> rr[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * T + t) * 8;
        rx[i] = load8<XB>(a.x, row * a.ld_x + c, a.cols - c);
        if constexpr (RB != 0) rr[i] = load8<RB>(a.res, row * a.ld_r + c, a.cols - c);
    }
    float h[P][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        widen8<XB>(rx[i], a.x_dtype == ZERO_BF16, h[i]);
        if constexpr (RB != 0) {
            float r[8];
            widen8<RB>(rr[i], a.r_dtype == ZERO_BF16, r);
#pragma unroll
            for (int k = 0; k < 8; ++k) h[i][k] += r[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += h[i][k];
    }
    if (a.h) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * T + t) * 8;
            store8(a.h, row * a.ld_h + c, a.cols - c, a.r_dtype, h[i]);
        }
    }
    const float mean = block_sum(sum, part[0]) * inv_cols;
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * T + t) * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            h[i][k] = c + k < a.cols ? h[i][k] - mean : 0.0f;
            ss = __builtin_fmaf(h[i][k], h[i][k], ss);
        }
    }
    ss = block_sum(ss, part[1]);
    const float rstd = 1.0f / sqrtf(ss * inv_cols + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    if (!a.y && !a.q) return;
    const int padded = (a.cols + 127) & ~127;
    const int blocks = padded / 128, blocks4 = (blocks + 3) & ~3;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * T + t) * 8;
        float w[8], b[8] = {};
        if (a.w_dtype == ZERO_F32) {
            widen8<4>(load8<4>(a.weight, c, a.cols - c), false, w);
            if (a.bias) widen8<4>(load8<4>(a.bias, c, a.cols - c), false, b);
        } else {
            widen8<2>(load8<2>(a.weight, c, a.cols - c), a.w_dtype == ZERO_BF16, w);
            if (a.bias) widen8<2>(load8<2>(a.bias, c, a.cols - c), a.w_dtype == ZERO_BF16, b);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)  // a NaN or inf rstd makes NaN of zeros
            h[i][k] = c + k < a.cols ? __builtin_fmaf(h[i][k] * rstd, w[k], b[k]) : 0.0f;
        if (a.y) store8(a.y, row * a.ld_y + c, a.cols - c, a.y_dtype, h[i]);
        if (a.q) {
            // 16 neighbouring lanes hold one block of 128
            const BlockScale s = block_scale(max16lanes(amax8(h[i])), a.fmt);
            if (c < padded)
                *reinterpret_cast<u32x2*>(a.q + row * a.ld_q + c) = pack8(h[i], s, a.fmt);
            const int bl = c / 128;
            if ((t & 15) == 0 && bl < blocks4)
                a.s[row * a.ld_s + bl] = static_cast<uint8_t>(bl < blocks ? s.byte : 127u);
        }
    }
}

template <int MAX_T, int P>
hipError_t norm_shape(const LayerNormArgs& a, hipStream_t stream) {
    const uint32_t block = static_cast<uint32_t>((a.cols + P * 512 - 1) / (P * 512) * 64);
    const bool x4 = a.x_dtype == ZERO_F32, r4 = a.r_dtype == ZERO_F32;
    auto run = [&](auto kernel) {
        return in_launches(a.rows, block, [&](int64_t first, uint32_t grid) {
            kernel<<<grid, block, 0, stream>>>(a, first);
            return hipGetLastError();
        });
    };
    if (!a.res)
        return x4 ? run(layernorm_kernel<MAX_T, P, 4, 0>) : run(layernorm_kernel<MAX_T, P, 2, 0>);
    if (r4)
        return x4 ? run(layernorm_kernel<MAX_T, P, 4, 4>) : run(layernorm_kernel<MAX_T, P, 2, 4>);
    return x4 ? run(layernorm_kernel<MAX_T, P, 4, 2>) : run(layernorm_kernel<MAX_T, P, 2, 2>);
}

}  // namespace

hipError_t launch_layernorm(const LayerNormArgs& a, hipStream_t stream) {
    const int c = a.cols;
    if (c <= 512) return norm_shape<64, 1>(a, stream);
    if (c <= 16384) return norm_shape<1024, 2>(a, stream);
    if (c <= 32768) return norm_shape<1024, 4>(a, stream);
    return norm_shape<1024, 8>(a, stream);
}

}  // namespace zero
