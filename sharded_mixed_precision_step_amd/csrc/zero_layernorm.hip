// Residual addition and layer norm.
//
// One pass over its arrays, bound by HBM: a row's elements stay in registers as
// fp32, between the sum for the mean, the sum of squares about that mean (two
// reductions, so that a row far from zero keeps its variance) and the outputs.
//
// 8192 x 4096 fp16 with an fp32 residual, h and an e4m3 output: 72 us, 5.1 TB/s, of 6.2
// that a large elementwise copy reaches.  16 rows: 4.5 us each in a graph, a launch, two
// trips to memory and two reductions.
#include "zero_device.h"
#include "zero_model_internal.h"

namespace zero {
namespace {

using namespace dev;

// Sum over a row's lanes: LPR neighbouring lanes of a wave, or the workgroup (LPR 0).
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
    if constexpr (LPR == 0) {
        return block_sum(v, part);
    } else {
#pragma unroll
        for (int d = 1; d < LPR; d *= 2) v += __shfl_xor(v, d);
        return v;
    }
}

// P packs of eight a lane.  LPR > 0: MAX_T lanes hold MAX_T / LPR rows.
template <int MAX_T, int LPR, int P, int XB, int RB, bool RAGGED>
__global__ __launch_bounds__(MAX_T) void layernorm_kernel(const LayerNormArgs a, int64_t first) {
    __shared__ float part[2][16];
    const int T = LPR == 0 ? static_cast<int>(blockDim.x) : LPR;
    const int t = LPR == 0 ? static_cast<int>(threadIdx.x) : threadIdx.x % LPR;
    const int64_t own = LPR == 0 ? first + blockIdx.x
                                 : (first + blockIdx.x) * (MAX_T / LPR) + threadIdx.x / LPR;
    const bool live = LPR == 0 || own < a.rows;
    const int64_t row = live ? own : a.rows - 1;  // lanes without a row go along
    const float inv_cols = 1.0f / static_cast<float>(a.cols);
    // of wide rows, four packs' loads at a time: more do not fit beside their values
    constexpr int kAtOnce = P > 4 ? 4 : P;
    float h[P][8];
    float sum = 0.0f;
#pragma unroll
    for (int i0 = 0; i0 < P; i0 += kAtOnce) {
        Raw8<XB> rx[kAtOnce];
        Raw8<RB == 0 ? 2 : RB> rr[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int c = ((i0 + i) * T + t) * 8;
            rx[i] = load8_row<XB, RAGGED>(a.x, row * a.ld_x, c, a.cols);
            if constexpr (RB != 0) rr[i] = load8_row<RB, RAGGED>(a.res, row * a.ld_r, c, a.cols);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int c = ((i0 + i) * T + t) * 8;
            float(&f)[8] = h[i0 + i];
            settle8<XB, RAGGED>(rx[i], c, a.cols);
            widen8<XB>(rx[i], a.x_dtype == ZERO_BF16, f);
            if constexpr (RB != 0) {
                float r[8];
                settle8<RB, RAGGED>(rr[i], c, a.cols);
                widen8<RB>(rr[i], a.r_dtype == ZERO_BF16, r);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] += r[k];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += f[k];
        }
        if constexpr (P > 4) __builtin_amdgcn_sched_barrier(0);
    }
    // on their way during the reductions
    constexpr bool kEarly = P <= 2;
    const bool w32 = a.w_dtype == ZERO_F32;
    Raw8<2> w16[kEarly ? P : 1], b16[kEarly ? P : 1];
    if (kEarly && !w32) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * T + t) * 8;
            w16[i] = load8_row<2, RAGGED>(a.weight, 0, c, a.cols);
            if (a.bias) b16[i] = load8_row<2, RAGGED>(a.bias, 0, c, a.cols);
        }
    }
    if (a.h) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * T + t) * 8;
            store8(a.h, row * a.ld_h + c, live ? a.cols - c : 0, a.r_dtype, h[i]);
        }
    }
    const float mean = row_sum<LPR>(sum, part[0]) * inv_cols;
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
    ss = row_sum<LPR>(ss, part[1]);
    const float rstd = 1.0f / sqrtf(ss * inv_cols + a.eps);
    if (t == 0 && live) {
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
        if (w32) {
            widen8<4>(load8<4>(a.weight, c, a.cols - c), false, w);
            if (a.bias) widen8<4>(load8<4>(a.bias, c, a.cols - c), false, b);
        } else {
            const bool bf16 = a.w_dtype == ZERO_BF16;
            Raw8<2> r = kEarly ? w16[kEarly ? i : 0] : load8_row<2, RAGGED>(a.weight, 0, c, a.cols);
            settle8<2, RAGGED>(r, c, a.cols);
            widen8<2>(r, bf16, w);
            if (a.bias) {
                r = kEarly ? b16[kEarly ? i : 0] : load8_row<2, RAGGED>(a.bias, 0, c, a.cols);
                settle8<2, RAGGED>(r, c, a.cols);
                widen8<2>(r, bf16, b);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)  // a NaN or inf rstd makes NaN of zeros
            h[i][k] = c + k < a.cols ? __builtin_fmaf(h[i][k] * rstd, w[k], b[k]) : 0.0f;
        if (a.y) store8(a.y, row * a.ld_y + c, live ? a.cols - c : 0, a.y_dtype, h[i]);
        if (a.q) {
            // 16 neighbouring lanes hold one block of 128
            const BlockScale s = block_scale(max16lanes(amax8(h[i])), a.fmt);
            if (c < padded && live)
                *reinterpret_cast<u32x2*>(a.q + row * a.ld_q + c) = pack8(h[i], s, a.fmt);
            const int bl = c / 128;
            // a row's first lanes fill the scales behind its last block
            uint8_t* at = a.s + row * a.ld_s;
            if ((t & 15) == 0 && bl < blocks && live) at[bl] = static_cast<uint8_t>(s.byte);
            if (i == 0 && t < blocks4 - blocks && live) at[blocks + t] = 127;
        }
        if constexpr (P > 4) __builtin_amdgcn_sched_barrier(0);
    }
}

template <int MAX_T, int LPR, int P, bool RAGGED>
hipError_t norm_shape(const LayerNormArgs& a, hipStream_t stream) {
    const uint32_t block = LPR != 0 ? MAX_T
                                    : static_cast<uint32_t>((a.cols + P * 512 - 1) / (P * 512) * 64);
    const int64_t per = LPR != 0 ? MAX_T / (LPR != 0 ? LPR : 1) : 1;
    const bool x4 = a.x_dtype == ZERO_F32, r4 = a.r_dtype == ZERO_F32;
    auto run = [&](auto kernel) {
        return in_launches((a.rows + per - 1) / per, block, [&](int64_t first, uint32_t grid) {
            kernel<<<grid, block, 0, stream>>>(a, first);
            return hipGetLastError();
        });
    };
    if (!a.res)
        return x4 ? run(layernorm_kernel<MAX_T, LPR, P, 4, 0, RAGGED>)
                  : run(layernorm_kernel<MAX_T, LPR, P, 2, 0, RAGGED>);
    if (r4)
        return x4 ? run(layernorm_kernel<MAX_T, LPR, P, 4, 4, RAGGED>)
                  : run(layernorm_kernel<MAX_T, LPR, P, 2, 4, RAGGED>);
    return x4 ? run(layernorm_kernel<MAX_T, LPR, P, 4, 2, RAGGED>)
              : run(layernorm_kernel<MAX_T, LPR, P, 2, 2, RAGGED>);
}

}  // namespace

// In fp16, with a residual and h: up to 1,024 columns a row is a few lanes' of one wave,
// whose reductions need no barrier (262144 x 128 124 us with a workgroup per row, 43 so);
// wider ones a workgroup's.  Rows that end inside a pack load their last eight elements
// (8192 x 1023 24 us by elements, 17 so; 8000 x 5001 93 and 77).  Above 16,384 columns a
// lane holds four or eight packs: 1024 x 32768 56 us; with eight it spills, 1024 x 65536
// 206 (84 without a residual).
hipError_t launch_layernorm(const LayerNormArgs& a, hipStream_t stream) {
    const int c = a.cols;
    if (c % 8 && c >= 8 && c <= 16384) {
        if (c <= 128) return norm_shape<256, 16, 1, true>(a, stream);
        if (c <= 256) return norm_shape<256, 32, 1, true>(a, stream);
        if (c <= 512) return norm_shape<256, 64, 1, true>(a, stream);
        if (c <= 1024) return norm_shape<256, 64, 2, true>(a, stream);
        return norm_shape<1024, 0, 2, true>(a, stream);
    }
    if (c <= 128) return norm_shape<256, 16, 1, false>(a, stream);
    if (c <= 256) return norm_shape<256, 32, 1, false>(a, stream);
    if (c <= 512) return norm_shape<256, 64, 1, false>(a, stream);
    if (c <= 1024) return norm_shape<256, 64, 2, false>(a, stream);
    if (c <= 16384) return norm_shape<1024, 0, 2, false>(a, stream);
    if (c <= 32768) return norm_shape<1024, 0, 4, false>(a, stream);
    return norm_shape<1024, 0, 8, false>(a, stream);
}

}  // namespace zero
