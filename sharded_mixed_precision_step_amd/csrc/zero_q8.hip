// A matrix in the 8-bit block layout, by rows, transposed, or both.
//
// One workgroup takes a 128 x 128 tile: the unit in which a block along a row
// and a block along a column are both whole, so one pass over src serves both
// outputs.  Bound by HBM.  By rows a block of 128 lies in 16 lanes' registers
// and its scale is found by shuffles.  For the transposed output the tile
// turns in LDS: it is written as loaded, read down its columns, and the 8-bit
// result is turned once more so that stores run along qt's rows.
#include "zero_device.h"
#include "zero_train_internal.h"

namespace zero {
namespace {

using namespace dev;

constexpr int kTile = 128;
constexpr int kThreads = 256;
constexpr int kSteps = kTile * kTile / (kThreads * 8);  // packs per lane

template <int B, bool ROWS, bool COLS>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const QuantizeArgs a,
                                                            uint32_t tiles_c) {
    const int t = threadIdx.x;
    const uint32_t tile_r = blockIdx.x / tiles_c;  // 32-bit: both fit
    const int64_t r0 = static_cast<int64_t>(tile_r) * kTile;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x - tile_r * tiles_c) * kTile;
    const void* src = a.src[a.ctl ? (a.ctl->cur & 1) : 0];
    const bool bf16 = a.dtype == ZERO_BF16;
    const int rows = static_cast<int>(a.rows - r0 < kTile ? a.rows - r0 : kTile);
    const int cols = static_cast<int>(a.cols - c0 < kTile ? a.cols - c0 : kTile);

    // lane t holds columns 8 * (t % 16) .. + 7 of rows t / 16 + 16 i
    const int c = t % 16 * 8;
    Raw8<B> raw[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int r = t / 16 + 16 * i;
        raw[i] = load8<B>(src, (r0 + r) * a.ld_src + c0 + c, r < rows ? cols - c : 0);
    }
    if constexpr (ROWS) {
        const int64_t b = c0 / kTile, blocks = (a.cols + 127) / 128;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = t / 16 + 16 * i;
            float f[8];
            widen8<B>(raw[i], bf16, f);
            const BlockScale s = block_scale(max16lanes(amax8(f)), a.fmt);
            if (r < rows) {
                *reinterpret_cast<u32x2*>(a.q + (r0 + r) * a.ld_q + c0 + c) = pack8(f, s, a.fmt);
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
        float v0[32], v1[32];
        uint32_t m0 = 0, m1 = 0;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            const uint8_t* at = lds + (32 * w + k) * kPitch + 2 * l * B;
            if constexpr (B == 4) {
                const u32x2 x = *reinterpret_cast<const u32x2*>(at);
                v0[k] = as_float(x[0]);
                v1[k] = as_float(x[1]);
            } else {
                const uint32_t x = *reinterpret_cast<const uint32_t*>(at);
                v0[k] = from16(x & 0xffffu, bf16);
                v1[k] = from16(x >> 16, bf16);
            }
            m0 = abs_bits(v0[k]) > m0 ? abs_bits(v0[k]) : m0;
            m1 = abs_bits(v1[k]) > m1 ? abs_bits(v1[k]) : m1;
        }
        amax[w][2 * l] = m0;
        amax[w][2 * l + 1] = m1;
        __syncthreads();  // also: every column has been read
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            m0 = amax[k][2 * l] > m0 ? amax[k][2 * l] : m0;
            m1 = amax[k][2 * l + 1] > m1 ? amax[k][2 * l + 1] : m1;
        }
        const BlockScale s0 = block_scale(m0, a.fmt), s1 = block_scale(m1, a.fmt);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const BlockScale& s = h ? s1 : s0;
            const float* v = h ? v1 : v0;
#pragma unroll
            for (int k = 0; k < 32; k += 16) {
                u32x4 out;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    out[j] = s.byte == 255u
                                 ? 0x7f7f7f7fu
                                 : pack4(v[k + 4 * j] * s.inv, v[k + 4 * j + 1] * s.inv,
                                         v[k + 4 * j + 2] * s.inv, v[k + 4 * j + 3] * s.inv,
                                         a.fmt);
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

template <int B>
void quantize_forms(const QuantizeArgs& a, dim3 grid, uint32_t tiles_c, hipStream_t stream) {
    if (!a.qt) quantize_kernel<B, true, false><<<grid, kThreads, 0, stream>>>(a, tiles_c);
    else if (!a.q) quantize_kernel<B, false, true><<<grid, kThreads, 0, stream>>>(a, tiles_c);
    else quantize_kernel<B, true, true><<<grid, kThreads, 0, stream>>>(a, tiles_c);
}

}  // namespace

int64_t quantize_blocks(int64_t rows, int64_t cols) {
    return (rows + kTile - 1) / kTile * ((cols + kTile - 1) / kTile);
}

hipError_t launch_q8_quantize(const QuantizeArgs& a, hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>(quantize_blocks(a.rows, a.cols)));
    const uint32_t tiles_c = static_cast<uint32_t>((a.cols + kTile - 1) / kTile);
    if (a.dtype == ZERO_F32) quantize_forms<4>(a, grid, tiles_c, stream);
    else quantize_forms<2>(a, grid, tiles_c, stream);
    return hipGetLastError();
}

}  // namespace zero
