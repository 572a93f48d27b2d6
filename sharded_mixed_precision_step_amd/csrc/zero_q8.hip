// A matrix in the 8-bit block layout, by rows, transposed, or both.
//
// One workgroup takes a 128 x 128 tile: the unit in which a block along a row
// and a block along a column are both whole, so one pass over src serves both
// outputs.  By rows a block of 128 lies in 16 lanes' registers and its scale is
// found by lane rotations.  For the transposed output the tile turns in LDS: it
// is written as loaded, read down its columns, and the 8-bit result is turned
// once more so that stores run along qt's rows.
//
// Bound by HBM: 14336 x 4096 fp16 in both forms takes 50 us, 4.7 TB/s, as a large
// copy (69 us with scaling and conversion as instructions of their own); by
// rows alone 36, transposed alone 38.
#include "zero_device.h"
#include "zero_train_internal.h"

namespace zero {
namespace {

using namespace dev;

constexpr int kTile = 128;
constexpr int kThreads = 256;
constexpr int kSteps = kTile * kTile / (kThreads * 8);  // packs per lane

typedef unsigned short v2u __attribute__((ext_vector_type(2)));

// Elementwise largest of two words' 16-bit halves, unsigned.
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2u, a),
                                                                  __builtin_bit_cast(v2u, b)));
}

// A lane's eight elements of a row: their largest magnitude, as the element
// type's bits (which order as the values do), and their 8-bit form.
template <int DT>
__device__ __forceinline__ uint32_t largest(const Raw8<DT == ZERO_F32 ? 4 : 2>& r) {
    if constexpr (DT == ZERO_F32) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = umax(m, r.v[k / 4][k % 4] & 0x7fffffffu);
        return m;
    } else {
        uint32_t m = r.v[0][0] & 0x7fff7fffu;
#pragma unroll
        for (int k = 1; k < 4; ++k) m = max_halves(m, r.v[0][k] & 0x7fff7fffu);
        return umax(m & 0xffffu, m >> 16);
    }
}
template <int DT>
__device__ __forceinline__ uint32_t fp32_bits(uint32_t magnitude) {
    return DT == ZERO_F32 ? magnitude : as_bits(from16(magnitude, DT == ZERO_BF16));
}
template <int DT, int FMT>
__device__ __forceinline__ u32x2 convert(const Raw8<DT == ZERO_F32 ? 4 : 2>& r,
                                         const BlockScale& s) {
    u32x2 out;
    if constexpr (DT == ZERO_F32) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            out[k] = pack4<FMT>(as_float(r.v[k][0]), as_float(r.v[k][1]), as_float(r.v[k][2]),
                                as_float(r.v[k][3]), s.scale);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            out[k] = pack4<FMT, DT == ZERO_BF16>(r.v[0][2 * k], r.v[0][2 * k + 1], s.scale);
    }
    return s.byte == 255u ? u32x2{kNan4, kNan4} : out;
}

template <int DT, int FMT, bool ROWS, bool COLS>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const QuantizeArgs a,
                                                            uint32_t tiles_c, uint32_t first) {
    constexpr int B = DT == ZERO_F32 ? 4 : 2;
    const int t = threadIdx.x;
    const uint32_t tile = first + blockIdx.x;  // 32-bit: all of them fit
    const uint32_t tile_r = tile / tiles_c;
    const int64_t r0 = static_cast<int64_t>(tile_r) * kTile;
    const int64_t c0 = static_cast<int64_t>(tile - tile_r * tiles_c) * kTile;
    const void* src = a.src[a.ctl ? (a.ctl->cur & 1) : 0];
    const int rows = static_cast<int>(a.rows - r0 < kTile ? a.rows - r0 : kTile);
    const int cols = static_cast<int>(a.cols - c0 < kTile ? a.cols - c0 : kTile);

    // lane t holds columns 8 * (t % 16) .. + 7 of rows t / 16 + 16 i
    const int c = t % 16 * 8;
    Raw8<B> raw[kSteps];
    if (rows == kTile && cols == kTile) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            raw[i] = load8<B>(src, (r0 + t / 16 + 16 * i) * a.ld_src + c0 + c, 8);
    } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = t / 16 + 16 * i;
            raw[i] = load8<B>(src, (r0 + r) * a.ld_src + c0 + c, r < rows ? cols - c : 0);
        }
    }
    if constexpr (ROWS) {
        const int64_t b = c0 / kTile, blocks = (a.cols + 127) / 128;
        uint32_t m[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) m[i] = max16lanes(largest<DT>(raw[i]));
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = t / 16 + 16 * i;
            const BlockScale s = block_scale(fp32_bits<DT>(m[i]), FMT);
            if (r < rows) {
                *reinterpret_cast<u32x2*>(a.q + (r0 + r) * a.ld_q + c0 + c) =
                    convert<DT, FMT>(raw[i], s);
                uint8_t* at = a.s + (r0 + r) * a.ld_s;
                if (t % 16 == 0) at[b] = static_cast<uint8_t>(s.byte);
                // the last block's lanes fill the scales behind it
                if (b == blocks - 1 && t % 16 >= 1 && t % 16 <= 3 && (b & 3) + t % 16 < 4)
                    at[b + t % 16] = 127;
            }
        }
    }
    if constexpr (COLS) {
        // the tile as loaded; a row's pitch of 128 elements and one pack keeps
        // the column reads of 64 lanes on neighbouring words
        constexpr int kPitch = kTile * B + 16;
        constexpr int kOutPitch = kTile + 16;
        __shared__ __attribute__((aligned(16))) uint8_t lds[kTile * kPitch];
        __shared__ uint32_t amax[4][kTile];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = t / 16 + 16 * i;
#pragma unroll
            for (int k = 0; k < B / 2; ++k)
                *reinterpret_cast<u32x4*>(lds + r * kPitch + c * B + 16 * k) = raw[i].v[k];
        }
        __syncthreads();
        // wave w, lane l: columns 2l and 2l + 1 of rows 32 w .. + 31
        const int w = t / 64, l = t % 64;
        uint32_t v[B / 2][32];  // 16-bit: both columns in a word
        uint32_t m0 = 0, m1 = 0, both = 0;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            const uint8_t* at = lds + (32 * w + k) * kPitch + 2 * l * B;
            if constexpr (B == 4) {
                const u32x2 x = *reinterpret_cast<const u32x2*>(at);
                v[0][k] = x[0];
                v[1][k] = x[1];
                m0 = umax(m0, x[0] & 0x7fffffffu);
                m1 = umax(m1, x[1] & 0x7fffffffu);
            } else {
                v[0][k] = *reinterpret_cast<const uint32_t*>(at);
                both = max_halves(both, v[0][k] & 0x7fff7fffu);
            }
        }
        if constexpr (B == 2) {
            m0 = both & 0xffffu;
            m1 = both >> 16;
        }
        amax[w][2 * l] = m0;
        amax[w][2 * l + 1] = m1;
        __syncthreads();  // also: every column has been read
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            m0 = umax(m0, amax[k][2 * l]);
            m1 = umax(m1, amax[k][2 * l + 1]);
        }
        const BlockScale s0 = block_scale(fp32_bits<DT>(m0), FMT);
        const BlockScale s1 = block_scale(fp32_bits<DT>(m1), FMT);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const BlockScale s = h ? s1 : s0;
#pragma unroll
            for (int k = 0; k < 32; k += 16) {
                u32x4 out;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = k + 4 * j;
                    if constexpr (B == 4) {
                        out[j] = pack4<FMT>(as_float(v[h][r]), as_float(v[h][r + 1]),
                                            as_float(v[h][r + 2]), as_float(v[h][r + 3]), s.scale);
                    } else {
                        // this column's halves of two rows in one word
                        constexpr uint32_t kLow = 0x05040100u, kHigh = 0x07060302u;
                        const uint32_t pick = h ? kHigh : kLow;
                        out[j] = pack4<FMT, DT == ZERO_BF16>(
                            __builtin_amdgcn_perm(v[0][r + 1], v[0][r], pick),
                            __builtin_amdgcn_perm(v[0][r + 3], v[0][r + 2], pick), s.scale);
                    }
                    if (s.byte == 255u) out[j] = kNan4;
                }
                *reinterpret_cast<u32x4*>(lds + (2 * l + h) * kOutPitch + 32 * w + k) = out;
            }
        }
        const int64_t b = r0 / kTile, blocks = (a.rows + 127) / 128;
        if (w == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (2 * l + h < cols) {
                    uint8_t* at = a.st + (c0 + 2 * l + h) * a.ld_st;
                    at[b] = static_cast<uint8_t>(h ? s1.byte : s0.byte);
                    if (b == blocks - 1)
                        for (int64_t k = b + 1; k & 3; ++k) at[k] = 127;
                }
            }
        }
        __syncthreads();
        // 8 lanes store one row of qt, 128 bytes
#pragma unroll
        for (int i = 0; i < kTile * kTile / (16 * kThreads); ++i) {
            const int j = t / 8 + 32 * i;
            if (j < cols)
                *reinterpret_cast<u32x4*>(a.qt + (c0 + j) * a.ld_qt + r0 + 16 * (t % 8)) =
                    *reinterpret_cast<const u32x4*>(lds + j * kOutPitch + 16 * (t % 8));
        }
    }
}

template <int DT, int FMT>
hipError_t quantize_forms(const QuantizeArgs& a, hipStream_t stream) {
    const uint32_t tiles_c = static_cast<uint32_t>((a.cols + kTile - 1) / kTile);
    auto run = [&](auto kernel) {
        return in_launches(quantize_blocks(a.rows, a.cols), kThreads,
                           [&](int64_t first, uint32_t grid) {
                               kernel<<<grid, kThreads, 0, stream>>>(
                                   a, tiles_c, static_cast<uint32_t>(first));
                               return hipGetLastError();
                           });
    };
    if (!a.qt) return run(quantize_kernel<DT, FMT, true, false>);
    if (!a.q) return run(quantize_kernel<DT, FMT, false, true>);
    return run(quantize_kernel<DT, FMT, true, true>);
}

template <int DT>
hipError_t quantize_type(const QuantizeArgs& a, hipStream_t stream) {
    return a.fmt == ZERO_E4M3 ? quantize_forms<DT, ZERO_E4M3>(a, stream)
                              : quantize_forms<DT, ZERO_E5M2>(a, stream);
}

}  // namespace

int64_t quantize_blocks(int64_t rows, int64_t cols) {
    return (rows + kTile - 1) / kTile * ((cols + kTile - 1) / kTile);
}

hipError_t launch_q8_quantize(const QuantizeArgs& a, hipStream_t stream) {
    if (a.dtype == ZERO_F32) return quantize_type<ZERO_F32>(a, stream);
    if (a.dtype == ZERO_F16) return quantize_type<ZERO_F16>(a, stream);
    return quantize_type<ZERO_BF16>(a, stream);
}

}  // namespace zero
