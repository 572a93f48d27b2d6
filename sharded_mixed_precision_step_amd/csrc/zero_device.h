// Device helpers of the training operators: element types, rows of any
// alignment, 8-bit blocks, reductions.  gfx950 only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_train.h"

namespace zero {
namespace dev {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// The same with an element's alignment: gfx950 loads and stores 16 bytes at
// any address, so rows need not be 16-byte aligned.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

// By value: clang's bit cast of a vector's element takes the vector's first.
__device__ __forceinline__ float as_float(uint32_t bits) { return __builtin_bit_cast(float, bits); }
__device__ __forceinline__ uint32_t as_bits(float v) { return __builtin_bit_cast(uint32_t, v); }

__device__ __forceinline__ float from16(uint32_t bits, bool bf16) {
    return bf16 ? as_float(bits << 16)
                : static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
}

// One rounding to nearest even; beyond the range of fp16: inf.
__device__ __forceinline__ uint32_t to16(float v, bool bf16) {
    return bf16 ? static_cast<uint32_t>(
                      __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)))
                : static_cast<uint32_t>(
                      __builtin_bit_cast(uint16_t, static_cast<_Float16>(v)));
}

__device__ __forceinline__ float load1(const void* p, int64_t i, int dtype) {
    if (dtype == ZERO_F32) return static_cast<const float*>(p)[i];
    return from16(static_cast<const uint16_t*>(p)[i], dtype == ZERO_BF16);
}

__device__ __forceinline__ void store1(void* p, int64_t i, int dtype, float v) {
    if (dtype == ZERO_F32)
        static_cast<float*>(p)[i] = v;
    else
        static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(to16(v, dtype == ZERO_BF16));
}

// Eight consecutive elements as loaded: 16 bytes of a 16-bit type, 32 of fp32.
template <int BYTES>
struct Raw8 {
    u32x4 v[BYTES == 4 ? 2 : 1];
};

// Elements i .. i + 7 of p, of which the first n (may be <= 0) exist; the
// others read as zero.
template <int BYTES>
__device__ __forceinline__ Raw8<BYTES> load8(const void* p, int64_t i, int n) {
    Raw8<BYTES> r;
    const char* at = static_cast<const char*>(p) + i * BYTES;
    if (n >= 8) {
#pragma unroll
        for (int k = 0; k < BYTES / 2; ++k)
            r.v[k] = reinterpret_cast<const u32x4_any*>(at)[k];
        return r;
    }
#pragma unroll
    for (int k = 0; k < BYTES / 2; ++k) r.v[k] = u32x4{0, 0, 0, 0};
    if (n > 0) {
        if constexpr (BYTES == 4) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(at);
#pragma unroll
            for (int k = 0; k < 7; ++k)
                if (k < n) r.v[k / 4][k % 4] = q[k];
        } else {
            const uint16_t* q = reinterpret_cast<const uint16_t*>(at);
#pragma unroll
            for (int k = 0; k < 7; ++k)
                if (k < n) r.v[0][k / 2] |= static_cast<uint32_t>(q[k]) << (16 * (k % 2));
        }
    }
    return r;
}

// Elements c .. c + 7 of the row of cols elements that starts at element `row` of
// p.  RAGGED, for eight columns or more: without a wait at the row's end, where
// the row's last eight are loaded, and settle8 moves them into place once they
// are needed.  What that loads of the pack before is dropped, so that it does not
// matter if its owner has written there meanwhile.
template <int BYTES, bool RAGGED>
__device__ __forceinline__ Raw8<BYTES> load8_row(const void* p, int64_t row, int c, int cols) {
    if constexpr (!RAGGED) return load8<BYTES>(p, row + c, cols - c);
    else return load8<BYTES>(p, row + (c < cols - 8 ? c : cols - 8), 8);
}
template <int BYTES, bool RAGGED>
__device__ __forceinline__ void settle8(Raw8<BYTES>& r, int c, int cols) {
    if constexpr (!RAGGED) return;
    const int back = c + 8 - cols;        // places that the elements lie too early
    if (__ballot(back > 0) == 0) return;  // a branch: most waves have no row's end
    constexpr int kWords = BYTES == 4 ? 8 : 4;
    const int words = BYTES == 4 ? back : back >> 1;
    uint32_t w[kWords];
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = r.v[k / 4][k % 4];
#pragma unroll
    for (int d = 1; d < kWords; d *= 2) {
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            const uint32_t from = k + d < kWords ? w[k + d < kWords ? k + d : 0] : 0;
            w[k] = words & d ? from : w[k];
        }
    }
    if constexpr (BYTES == 2) {
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            const uint32_t above = k + 1 < kWords ? w[k + 1 < kWords ? k + 1 : 0] : 0;
            w[k] = back & 1 ? w[k] >> 16 | above << 16 : w[k];
        }
    }
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
        const uint32_t moved = back < 8 ? w[k] : 0;
        r.v[k / 4][k % 4] = back > 0 ? moved : r.v[k / 4][k % 4];
    }
}

// Waits for a load: what stands behind it may be written where it read.
template <int BYTES>
__device__ __forceinline__ void arrived(const Raw8<BYTES>& r) {
#pragma unroll
    for (int k = 0; k < (BYTES == 4 ? 2 : 1); ++k) asm volatile("" ::"v"(r.v[k]) : "memory");
}

template <int BYTES>
__device__ __forceinline__ void widen8(const Raw8<BYTES>& r, bool bf16, float (&f)[8]) {
    if constexpr (BYTES == 4) {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = as_float(r.v[k / 4][k % 4]);
    } else {
        if (bf16) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                f[k] = as_float(k % 2 ? r.v[0][k / 2] & 0xffff0000u : r.v[0][k / 2] << 16);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = from16(r.v[0][k / 2] >> (16 * (k % 2)), false);
        }
    }
}

// Stores the first n (at most 8) of f as elements i .. of p.
template <bool NT = false>
__device__ __forceinline__ void store8(void* p, int64_t i, int n, int dtype, const float (&f)[8]) {
    if (n <= 0) return;
    if (n >= 8) {
        if (dtype == ZERO_F32) {
            u32x4_any* at = reinterpret_cast<u32x4_any*>(static_cast<float*>(p) + i);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                u32x4 v;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = as_bits(f[4 * k + j]);
                if constexpr (NT) __builtin_nontemporal_store(v, at + k);
                else at[k] = v;
            }
        } else {
            u32x4 v;
            if (dtype == ZERO_BF16) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = to16(f[2 * k], true) | to16(f[2 * k + 1], true) << 16;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = to16(f[2 * k], false) | to16(f[2 * k + 1], false) << 16;
            }
            u32x4_any* at = reinterpret_cast<u32x4_any*>(static_cast<uint16_t*>(p) + i);
            if constexpr (NT) __builtin_nontemporal_store(v, at);
            else *at = v;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 7; ++k)
        if (k < n) store1(p, i + k, dtype, f[k]);
}

// ---- 8-bit blocks --------------------------------------------------------

struct BlockScale {
    float scale;   // 2^e
    uint32_t byte; // e + 127, or 255
};

// The scale of a block whose largest magnitude has these fp32 bits (sign
// cleared).  Both 8-bit types' largest value is 1.75 * 2^top (448 = 1.75 * 2^8,
// 57344 = 1.75 * 2^15), so the smallest e with amax <= 1.75 * 2^(top + e) is
// amax's own exponent less top, one more if its mantissa is above 1.75.  A
// NaN's or inf's bits compare above every finite value's.
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits, int fmt) {
    const int top = fmt == ZERO_E4M3 ? 8 : 15;
    int e = static_cast<int>(amax_bits >> 23) - 127 - top + ((amax_bits & 0x7fffffu) > 0x600000u);
    e = e < -127 ? -127 : e;
    if (amax_bits == 0) e = 0;
    BlockScale r;
    r.byte = static_cast<uint32_t>(e + 127);
    r.scale = as_float(r.byte == 0 ? 0x400000u : r.byte << 23);
    if (amax_bits >= 0x7f800000u) r.byte = 255u;
    return r;
}

typedef short v2s __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

// Four values over 2^e as 8-bit floats, rounded to nearest even: one
// instruction a pair divides, rounds and packs.
template <int FMT>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d, float scale) {
    v2s r = {0, 0};
    if constexpr (FMT == ZERO_E4M3) {
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, scale, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, scale, true);
    } else {
        r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(r, a, b, scale, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(r, c, d, scale, true);
    }
    return __builtin_bit_cast(uint32_t, r);
}

// The same of two words of two 16-bit values each.
template <int FMT, bool BF16>
__device__ __forceinline__ uint32_t pack4(uint32_t ab, uint32_t cd, float scale) {
    v2s r = {0, 0};
    if constexpr (BF16) {
        const v2b x = __builtin_bit_cast(v2b, ab), y = __builtin_bit_cast(v2b, cd);
        if constexpr (FMT == ZERO_E4M3) {
            r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, x, scale, false);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, y, scale, true);
        } else {
            r = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(r, x, scale, false);
            r = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(r, y, scale, true);
        }
    } else {
        const v2h x = __builtin_bit_cast(v2h, ab), y = __builtin_bit_cast(v2h, cd);
        if constexpr (FMT == ZERO_E4M3) {
            r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, x, scale, false);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, y, scale, true);
        } else {
            r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(r, x, scale, false);
            r = __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(r, y, scale, true);
        }
    }
    return __builtin_bit_cast(uint32_t, r);
}

constexpr uint32_t kNan4 = 0x7f7f7f7fu;  // four NaNs in both types

__device__ __forceinline__ u32x2 pack8(const float (&f)[8], const BlockScale& s, int fmt) {
    if (s.byte == 255u) return u32x2{kNan4, kNan4};
    if (fmt == ZERO_E4M3)
        return u32x2{pack4<ZERO_E4M3>(f[0], f[1], f[2], f[3], s.scale),
                     pack4<ZERO_E4M3>(f[4], f[5], f[6], f[7], s.scale)};
    return u32x2{pack4<ZERO_E5M2>(f[0], f[1], f[2], f[3], s.scale),
                 pack4<ZERO_E5M2>(f[4], f[5], f[6], f[7], s.scale)};
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return as_bits(v) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t amax8(const float (&f)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = umax(m, abs_bits(f[k]));
    return m;
}

// The largest of 16 neighbouring lanes', by rotations of the 16.
__device__ __forceinline__ uint32_t max16lanes(uint32_t m) {
    m = umax(m, __builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x121, 0xf, 0xf, true));
    m = umax(m, __builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x122, 0xf, 0xf, true));
    m = umax(m, __builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x124, 0xf, 0xf, true));
    return umax(m, __builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x128, 0xf, 0xf, true));
}

// ---- reductions ----------------------------------------------------------

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

// Sum over a workgroup of up to 1,024 threads, whole waves; `part` holds a float
// per wave.  The same value, summed in the same order, on every thread.  Two
// calls may not share `part` without a barrier between them.
__device__ __forceinline__ float block_sum(float v, float* part) {
    v = wave_sum(v);
    const int waves = static_cast<int>(blockDim.x >> 6);
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = part[0];
    for (int w = 1; w < waves; ++w) s += part[w];
    return s;
}

}  // namespace dev
}  // namespace zero
