// Activations with 8-bit checkpoints, and their gradients from them.
//
// Elementwise but for the largest magnitude of each block of 128, which is 16
// neighbouring lanes' (eight elements a lane), and bound by HBM: a lane holds one
// pack of each array.  8192 x 14336 fp16 gated, e4m3 output and checkpoints: 153 to 163
// us, 5.1 to 5.4 TB/s, the vector units busy in three quarters of the cycles; its gradient
// with y once more 198 to 203 us, 5.8 to 6.0 TB/s, half of them.  1003 x 5001 bf16, GELU:
// 8.2 us for what a large copy's rate would carry in 4.1, a wave and a half for each place,
// one trip to memory each.
#include "zero_device.h"
#include "zero_model_internal.h"

namespace zero {
namespace {

using namespace dev;

constexpr int kLanes = 256;
constexpr float kLog2e = 1.4426950408889634f;

// What an activation is made of: f(g) = g * s, f'(g) = s + g * d.
struct Slope {
    float s, d;
};

// 1 / (1 + exp(-v)) and 1 less that: exp(-|v|) neither overflows nor cancels.  The larger
// end is good to 3 half units of fp32's last place (2^-24).  The smaller has the error of
// the exponent's product, which grows with |v|: SiLU's values are off by at most 10 half
// units down to -9, 18 to -19, 32 to -33, 66 to -87; and it is 0 below -87.3, where fp32's
// normal range ends.
__device__ __forceinline__ Slope sigmoid(float v) {
    const float e = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e);
    const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
    return v < 0.0f ? Slope{small, big} : Slope{big, small};
}

// DERIVED: the derivative is asked for too.
template <int KIND, bool DERIVED>
__device__ __forceinline__ Slope slope(float g) {
    if constexpr (KIND == ZERO_SILU && !DERIVED) {
        // exp(-g) may overflow; below -87.33, where f is under 1.03e-36, s is 0, as the
        // other form's.  (By the form with both ends 8192 x 14336 162 us, 158 so.)
        return {__builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * g)), 0.0f};
    } else if constexpr (KIND == ZERO_SILU) {
        const Slope p = sigmoid(g);
        return {p.s, p.s * p.d};
    } else if constexpr (KIND == ZERO_GELU) {
        // With x = |g|: Phi(-x) = exp(-x^2 / 2) t P(t), t = 1 / (1 + x / 4), P a
        // polynomial fitted to the scaled complementary error function (itself to 5e-8 of
        // the value); Phi(x) = 1 - Phi(-x).  So small values of Phi do not cancel, and the
        // derivative's exponential serves both.  The exponent's products are rounded at
        // x^2's size, which is most of the error: at most 9 half units (2^-24) of the value
        // down to -2.2, 17 to -4.3, 55 to -8.7, 133 to -13; 6 above 0.  (With the library's
        // complementary error function: 8192 x 2048 fp16 30 us, 21 so.)
        const float x = fabsf(g), t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.25f, x, 1.0f));
        const float e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * x * x);
        float m = 0.019782092f;
        m = __builtin_fmaf(m, t, -0.080877684f);
        m = __builtin_fmaf(m, t, 0.09559778f);
        m = __builtin_fmaf(m, t, -0.031718224f);
        m = __builtin_fmaf(m, t, 0.063699536f);
        m = __builtin_fmaf(m, t, 0.058974996f);
        m = __builtin_fmaf(m, t, 0.08160314f);
        m = __builtin_fmaf(m, t, 0.09346635f);
        m = __builtin_fmaf(m, t, 0.09973643f);
        m = __builtin_fmaf(m, t, 0.099735565f);
        const float tail = e * t * m;
        return {g < 0.0f ? tail : 1.0f - tail, 0.39894228f * e};
    } else {
        // (1 + tanh u) / 2 = 1 / (1 + exp(-2u)), u = k (g + 0.044715 g^3); both
        // are 0 or 1 long before 64, and g^3 stays in range.  Off by 2u's roundings too, at
        // most 25 half units down to -2.7, 57 to -4.7, 128 to -6.7, 202 to -8; 4 above 0
        constexpr float k2 = 1.5957691f, kCube = 0.044715f;
        const float x = g != g ? g : fminf(fmaxf(g, -64.0f), 64.0f), xx = x * x;
        const Slope p = sigmoid(k2 * x * __builtin_fmaf(kCube, xx, 1.0f));
        return {p.s, p.s * p.d * (k2 * __builtin_fmaf(3.0f * kCube, xx, 1.0f))};
    }
}

// Where a workgroup's lanes are: rows of `lanes` lanes each (a power of two from
// 16 to 256), 8 columns a lane; padded columns have lanes too.
struct Place {
    int64_t row;
    int64_t c;
    bool live;    // the row exists and the column is inside the padded row
    int n;        // elements of the pack, may be <= 0
};
__device__ __forceinline__ Place place(int64_t first, int shift, uint32_t slices, int64_t rows,
                                       int64_t cols) {
    const uint32_t block = static_cast<uint32_t>(first + blockIdx.x);  // all of them fit
    const uint32_t group = block / slices;
    Place p;
    p.row = static_cast<int64_t>(group) * (kLanes >> shift) + (threadIdx.x >> shift);
    p.c = (static_cast<int64_t>(block - group * slices) << shift |
           (threadIdx.x & ((1 << shift) - 1))) * 8;
    const int64_t padded = (cols + 127) & ~int64_t{127}, left = cols - p.c;
    p.live = p.row < rows && p.c < padded;
    p.n = p.live ? static_cast<int>(left < 8 ? left : 8) : 0;
    return p;
}

// f in the q8 layout; all 16 lanes of a block call it.
__device__ __forceinline__ void put_q8(uint8_t* q, int64_t ld_q, uint8_t* s, int64_t ld_s, int fmt,
                                       const Place& p, int64_t cols, const float (&f)[8]) {
    const BlockScale b = block_scale(max16lanes(amax8(f)), fmt);
    if (!p.live) return;
    *reinterpret_cast<u32x2*>(q + p.row * ld_q + p.c) = pack8(f, b, fmt);
    const int64_t block = p.c / 128, blocks = (cols + 127) / 128;
    const int lane = threadIdx.x & 15;
    uint8_t* at = s + p.row * ld_s;
    if (lane == 0) at[block] = static_cast<uint8_t>(b.byte);
    // the last block's lanes fill the scales behind it
    if (block == blocks - 1 && lane >= 1 && lane <= 3 && (block & 3) + lane < 4)
        at[block + lane] = 127;
}

template <int KIND, int XB, bool UP>
__global__ __launch_bounds__(kLanes) void act_kernel(const ActArgs a, int64_t first, int shift,
                                                     uint32_t slices) {
    const Place p = place(first, shift, slices, a.rows, a.cols);
    const bool bf16 = a.x_dtype == ZERO_BF16;
    const Raw8<XB> rg = load8<XB>(a.gate, p.row * a.ld_g + p.c, p.n);
    Raw8<XB> ru;
    if constexpr (UP) ru = load8<XB>(a.up, p.row * a.ld_u + p.c, p.n);
    float g[8], u[8];
    widen8<XB>(rg, bf16, g);
    if constexpr (UP) widen8<XB>(ru, bf16, u);
    if (a.gate_q) put_q8(a.gate_q, a.ld_gq, a.gate_s, a.ld_gs, a.ck_fmt, p, a.cols, g);
    if constexpr (UP) {
        if (a.up_q) put_q8(a.up_q, a.ld_uq, a.up_s, a.ld_us, a.ck_fmt, p, a.cols, u);
    }
    if (!a.y && !a.q) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        g[k] = g[k] * slope<KIND, false>(g[k]).s;
        if constexpr (UP) g[k] *= u[k];
    }
    if (a.y) store8(a.y, p.row * a.ld_y + p.c, p.n, a.y_dtype, g);
    if (a.q) put_q8(a.q, a.ld_q, a.s, a.ld_s, a.fmt, p, a.cols, g);
}

// Eight values of a checkpoint.
template <int FMT>
__device__ __forceinline__ void from_q8(u32x2 q, uint32_t byte, float (&f)[8]) {
    typedef float v2f __attribute__((ext_vector_type(2)));
    const float scale = as_float(byte == 0 ? 0x400000u : byte == 255u ? 0x7fc00000u : byte << 23);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        v2f lo, hi;
        if constexpr (FMT == ZERO_E4M3) {
            lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q[k]), false);
            hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q[k]), true);
        } else {
            lo = __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(q[k]), false);
            hi = __builtin_amdgcn_cvt_pk_f32_bf8(static_cast<int>(q[k]), true);
        }
        f[4 * k] = lo[0] * scale;
        f[4 * k + 1] = lo[1] * scale;
        f[4 * k + 2] = hi[0] * scale;
        f[4 * k + 3] = hi[1] * scale;
    }
}

template <int KIND, int FMT, int DB, bool UP>
__global__ __launch_bounds__(kLanes) void act_backward_kernel(const ActBackwardArgs a,
                                                              int64_t first, int shift,
                                                              uint32_t slices) {
    const Place p = place(first, shift, slices, a.rows, a.cols);
    if (p.n <= 0) return;
    const int64_t block = p.c / 128;
    const u32x2 qg = *reinterpret_cast<const u32x2*>(a.gate_q + p.row * a.ld_gq + p.c);
    const uint32_t sg = a.gate_s[p.row * a.ld_gs + block];
    u32x2 qu;
    uint32_t su = 127u;
    if constexpr (UP) {
        qu = *reinterpret_cast<const u32x2*>(a.up_q + p.row * a.ld_uq + p.c);
        su = a.up_s[p.row * a.ld_us + block];
    }
    float dy[8], g[8], u[8];
    widen8<DB>(load8<DB>(a.dy, p.row * a.ld_dy + p.c, p.n), a.dy_dtype == ZERO_BF16, dy);
    from_q8<FMT>(qg, sg, g);
    if constexpr (UP) from_q8<FMT>(qu, su, u);
    float dup[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const Slope v = slope<KIND, true>(g[k]);
        float f = g[k] * v.s, d = dy[k] * __builtin_fmaf(g[k], v.d, v.s);
        if constexpr (UP) {
            dup[k] = dy[k] * f;
            d *= u[k];
            f *= u[k];
        }
        dy[k] = d;
        g[k] = f;
    }
    store8(a.dgate, p.row * a.ld_dg + p.c, p.n, a.dx_dtype, dy);
    if constexpr (UP) store8(a.dup, p.row * a.ld_du + p.c, p.n, a.dx_dtype, dup);
    if (a.y) store8(a.y, p.row * a.ld_y + p.c, p.n, a.y_dtype, g);
}

// Lanes per row, as a power of two: what the padded row needs, up to a workgroup.
int lanes_shift(int64_t cols) {
    int shift = 4;
    while (shift < 8 && (int64_t{8} << shift) < cols) ++shift;
    return shift;
}
int64_t row_slices(int64_t cols) {
    const int64_t span = int64_t{8} << lanes_shift(cols);
    return (cols + span - 1) / span;
}

template <class Args, class Kernel>
hipError_t run(Kernel kernel, const Args& a, hipStream_t stream) {
    const int shift = lanes_shift(a.cols);
    const uint32_t slices = static_cast<uint32_t>(row_slices(a.cols));  // below act_blocks
    return in_launches(act_blocks(a.rows, a.cols), kLanes, [&](int64_t first, uint32_t grid) {
        kernel<<<grid, kLanes, 0, stream>>>(a, first, shift, slices);
        return hipGetLastError();
    });
}

template <int KIND>
hipError_t act_kind(const ActArgs& a, hipStream_t stream) {
    if (a.x_dtype == ZERO_F32)
        return a.up ? run(act_kernel<KIND, 4, true>, a, stream)
                    : run(act_kernel<KIND, 4, false>, a, stream);
    return a.up ? run(act_kernel<KIND, 2, true>, a, stream)
                : run(act_kernel<KIND, 2, false>, a, stream);
}

template <int KIND, int FMT>
hipError_t backward_format(const ActBackwardArgs& a, hipStream_t stream) {
    if (a.dy_dtype == ZERO_F32)
        return a.up_q ? run(act_backward_kernel<KIND, FMT, 4, true>, a, stream)
                      : run(act_backward_kernel<KIND, FMT, 4, false>, a, stream);
    return a.up_q ? run(act_backward_kernel<KIND, FMT, 2, true>, a, stream)
                  : run(act_backward_kernel<KIND, FMT, 2, false>, a, stream);
}

template <int KIND>
hipError_t backward_kind(const ActBackwardArgs& a, hipStream_t stream) {
    return a.ck_fmt == ZERO_E4M3 ? backward_format<KIND, ZERO_E4M3>(a, stream)
                                 : backward_format<KIND, ZERO_E5M2>(a, stream);
}

}  // namespace

int64_t act_blocks(int64_t rows, int64_t cols) {
    const int64_t per = kLanes >> lanes_shift(cols);
    return (rows + per - 1) / per * row_slices(cols);
}

hipError_t launch_act(const ActArgs& a, hipStream_t stream) {
    if (a.kind == ZERO_SILU) return act_kind<ZERO_SILU>(a, stream);
    if (a.kind == ZERO_GELU) return act_kind<ZERO_GELU>(a, stream);
    return act_kind<ZERO_GELU_TANH>(a, stream);
}

hipError_t launch_act_backward(const ActBackwardArgs& a, hipStream_t stream) {
    if (a.kind == ZERO_SILU) return backward_kind<ZERO_SILU>(a, stream);
    if (a.kind == ZERO_GELU) return backward_kind<ZERO_GELU>(a, stream);
    return backward_kind<ZERO_GELU_TANH>(a, stream);
}

}  // namespace zero
