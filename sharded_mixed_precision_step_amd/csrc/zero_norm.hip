// Residual addition and root-mean-square norm.
//
// One pass over its arrays, bound by HBM: a row's elements stay in registers
// between the reduction over the row and the outputs that need it.  A row is
// held by one workgroup, eight elements (one 16-byte pack of a 16-bit type) per
// lane and step, so the workgroup size follows from the row's length: one wave
// up to 1,024 columns, four waves at 4,096.
//
// 8192 x 4096, fp16 with an fp32 residual, h, an e4m3 output and rstd: 69 us, 5.3
// TB/s, above what a large copy reaches (4.8).  16 rows: 4.4 us, two trips to
// memory and a launch.  Above 32,768 columns a lane's 64 fp32 values and its packs
// do not fit its 128 registers, and what is spilled goes through memory: 1024 x
// 65536 fp16 78 us, 3.5 TB/s.  Rows of less than 512 columns leave lanes of their
// wave without elements: 262144 x 128 79 us, 1.7 TB/s; 65536 x 256 24 us, 2.8.
#include "zero_device.h"
#include "zero_train_internal.h"

namespace zero {
namespace {

using namespace dev;

template <int MAX_T, int P, int XB, int RB, bool RAGGED>
__global__ __launch_bounds__(MAX_T) void rmsnorm_kernel(const NormArgs a, int64_t first) {
    __shared__ float part[16];
    const int T = static_cast<int>(blockDim.x);
    const int64_t row = first + blockIdx.x;
    const int t = threadIdx.x;
    Raw8<XB> rx[P];
    Raw8<RB == 0 ? 2 : RB> rr[P];
    Raw8<2> w16[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * T + t) * 8;
        rx[i] = load8_row<XB, RAGGED>(a.x, row * a.ld_x, c, a.cols);
        if constexpr (RB != 0) rr[i] = load8_row<RB, RAGGED>(a.res, row * a.ld_r, c, a.cols);
    }
    const bool w32 = a.w_dtype == ZERO_F32;
    if (!w32) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * T + t) * 8;
            w16[i] = load8_row<2, RAGGED>(a.weight, 0, c, a.cols);
        }
    }
    float h[P][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * T + t) * 8;
        settle8<XB, RAGGED>(rx[i], c, a.cols);
        widen8<XB>(rx[i], a.x_dtype == ZERO_BF16, h[i]);
        if constexpr (RB != 0) {
            float r[8];
            settle8<RB, RAGGED>(rr[i], c, a.cols);
            widen8<RB>(rr[i], a.r_dtype == ZERO_BF16, r);
#pragma unroll
            for (int k = 0; k < 8; ++k) h[i][k] += r[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = __builtin_fmaf(h[i][k], h[i][k], ss);
    }
    if (a.h) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * T + t) * 8;
            store8(a.h, row * a.ld_h + c, a.cols - c, a.r_dtype, h[i]);
        }
    }
    ss = block_sum(ss, part);
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.cols) + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    if (!a.y && !a.q) return;
    const int padded = (a.cols + 127) & ~127;
    const int blocks = padded / 128, blocks4 = (blocks + 3) & ~3;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * T + t) * 8;
        float w[8];
        if (w32) {
            const Raw8<4> r = load8<4>(a.weight, c, a.cols - c);
            widen8<4>(r, false, w);
        } else {
            settle8<2, RAGGED>(w16[i], c, a.cols);
            widen8<2>(w16[i], a.w_dtype == ZERO_BF16, w);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) h[i][k] = h[i][k] * rstd * w[k];
        // a NaN or inf rstd makes NaN of the zeros behind the row's end
        if (c + 8 > a.cols) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c + k >= a.cols) h[i][k] = 0.0f;
        }
        if (a.y) store8(a.y, row * a.ld_y + c, a.cols - c, a.y_dtype, h[i]);
        if (a.q) {
            // 16 neighbouring lanes hold one block of 128
            const BlockScale s = block_scale(max16lanes(amax8(h[i])), a.fmt);
            if (c < padded)
                *reinterpret_cast<u32x2*>(a.q + row * a.ld_q + c) = pack8(h[i], s, a.fmt);
            const int b = c / 128;
            if ((t & 15) == 0 && b < blocks4)
                a.s[row * a.ld_s + b] = static_cast<uint8_t>(b < blocks ? s.byte : 127u);
        }
    }
}

template <int MAX_T, int P, bool RAGGED = false>
hipError_t norm_shape(const NormArgs& a, hipStream_t stream) {
    const uint32_t block = static_cast<uint32_t>((a.cols + P * 512 - 1) / (P * 512) * 64);
    const bool x4 = a.x_dtype == ZERO_F32, r4 = a.r_dtype == ZERO_F32;
    auto run = [&](auto kernel) {
        return in_launches(a.rows, block, [&](int64_t first, uint32_t grid) {
            kernel<<<grid, block, 0, stream>>>(a, first);
            return hipGetLastError();
        });
    };
    if (!a.res)
        return x4 ? run(rmsnorm_kernel<MAX_T, P, 4, 0, RAGGED>)
                  : run(rmsnorm_kernel<MAX_T, P, 2, 0, RAGGED>);
    if (r4)
        return x4 ? run(rmsnorm_kernel<MAX_T, P, 4, 4, RAGGED>)
                  : run(rmsnorm_kernel<MAX_T, P, 2, 4, RAGGED>);
    return x4 ? run(rmsnorm_kernel<MAX_T, P, 4, 2, RAGGED>)
              : run(rmsnorm_kernel<MAX_T, P, 2, 2, RAGGED>);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t stream) {
    const int c = a.cols;
    // Rows that end inside a pack: a tail loaded by elements stops its wave for
    // each array in turn (fp16, 16 x 4095 6.2 us, now 4.9; 8192 x 1023 18, 14;
    // 8192 x 4097 with an fp32 residual 73, 74; rows without a tail take 47 us as
    // they are and 53 this way, 8000 x 5000).  Above 16,384 columns it is one wave
    // of many.
    if (c % 8 && c >= 8 && c <= 16384) {
        if (c <= 512) return norm_shape<64, 1, true>(a, stream);
        return norm_shape<1024, 2, true>(a, stream);
    }
    if (c <= 512) return norm_shape<64, 1>(a, stream);
    if (c <= 16384) return norm_shape<1024, 2>(a, stream);
    if (c <= 32768) return norm_shape<1024, 4>(a, stream);
    return norm_shape<1024, 8>(a, stream);
}

}  // namespace zero
