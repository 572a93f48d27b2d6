// Distillation from a teacher's top logits: loss and gradient.
//
// One workgroup per row.  The student's row goes by once for the running
// maximum and sum of its softmax (fp32, from a finite start so that a row of
// -inf stays countable) and once more for the gradient.  The teacher's entries,
// at most 1,024, sit in LDS.  The gradient is first written as coef * q_v for
// the whole row; behind a barrier the entries' places are written again with
// their p_j taken off, each computed from the logit read before anything was
// written, so that one rounding is made and the gradient may take the
// logits' place.
#include "zero_device.h"
#include "zero_train_internal.h"

namespace zero {
namespace {

using namespace dev;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;

// exp(x) for x * log2(e) formed by the caller
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

struct Stat {
    float m, s;  // running maximum, sum of exp2((x - m) * c)
};

__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
    const float m = fmaxf(a.m, b.m);
    return {m, a.s * exp2_fast((a.m - m) * c) + b.s * exp2_fast((b.m - m) * c)};
}

// One teacher entry per thread and step; T threads.
constexpr int kT = 1024;

struct Entries {
    int32_t idx[ZERO_DISTILL_MAX_TOP];
    float p[ZERO_DISTILL_MAX_TOP];
    float x[ZERO_DISTILL_MAX_TOP];  // the student's logit there, times 1
    float red[2 * (kT / 64)];
    int32_t bad;
};

__device__ __forceinline__ float block_max(float v, float* part) {
    v = wave_max(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = part[0];
#pragma unroll
    for (int w = 1; w < kT / 64; ++w) s = fmaxf(s, part[w]);
    return s;
}

__device__ __forceinline__ float block_add(float v, float* part) {
    __syncthreads();
    return block_sum(v, part);
}

template <int B, DistillMode MODE>
__global__ __launch_bounds__(kT) void distill_kernel(const DistillArgs a) {
    __shared__ Entries e;
    const int t = threadIdx.x;
    const int64_t row = blockIdx.x;
    const bool bf16 = a.dtype == ZERO_BF16;
    const float weight = a.weight ? a.weight[row] : 1.0f;
    const int vocab = static_cast<int>(a.vocab);
    const char* x = static_cast<const char*>(a.logits) + row * a.ld * B;
    char* g = static_cast<char*>(a.grad) + row * a.ld_grad * B;
    if (weight == 0.0f) {
        if (MODE != kDistillBackward && t == 0) {
            if (a.loss) a.loss[row] = 0.0f;
            if (a.lse) a.lse[row] = 0.0f;
        }
        if (MODE != kDistillForward) {
            const float zero[8] = {};
            for (int v = 8 * t; v < vocab; v += 8 * kT) store8(g, v, vocab - v, a.dtype, zero);
        }
        return;
    }
    if (t == 0) e.bad = 0;
    __syncthreads();
    // entries, at most one per thread
    const float inv_tau = 1.0f / a.tau;
    float tl = kLowest;
    bool have = false;
    int32_t idx = -1;
    if (t < a.top) {
        const int64_t at = row * a.ld_top + t;
        const int64_t i = a.index_bytes == 8 ? static_cast<const int64_t*>(a.index)[at]
                                             : static_cast<const int32_t*>(a.index)[at];
        if (i >= vocab) {
            e.bad = 1;
        } else if (i >= 0) {
            const float v = load1(a.top_logit, at, a.top_dtype);
            if (!(v < __builtin_inff())) {
                e.bad = 1;  // NaN or +inf
            } else if (v > -__builtin_inff()) {
                have = true;
                tl = v / a.tau;
            }
            idx = static_cast<int32_t>(i);
        }
        e.idx[t] = idx;
        e.x[t] = idx >= 0 ? load1(x, idx, a.dtype) : 0.0f;
    }
    const float tmax = block_max(tl, e.red);
    const float pe = have ? expf(tl - tmax) : 0.0f;
    const float psum = block_add(pe, e.red);
    const float p = have ? pe / psum : 0.0f;
    if (t < a.top) e.p[t] = p;
    const bool empty = psum == 0.0f;

    const float c = kLog2e * inv_tau;
    float lse, m = 0.0f, log2s = 0.0f;
    if (MODE != kDistillBackward) {
        Stat st = {kLowest, 0.0f};
        for (int v = 8 * t; v < vocab; v += 8 * kT) {
            const Raw8<B> r = load8<B>(x, v, vocab - v);
            float f[8];
            widen8<B>(r, bf16, f);
            if (v + 8 > vocab) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (v + k >= vocab) f[k] = -__builtin_inff();
            }
            float pm = st.m;
#pragma unroll
            for (int k = 0; k < 8; ++k) pm = fmaxf(pm, f[k]);
            st.s *= exp2_fast((st.m - pm) * c);
            st.m = pm;
#pragma unroll
            for (int k = 0; k < 8; ++k) st.s += exp2_fast((f[k] - pm) * c);
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const Stat o = {__shfl_xor(st.m, d), __shfl_xor(st.s, d)};
            st = join(st, o, c);
        }
        __syncthreads();
        if ((t & 63) == 0) {
            e.red[t >> 6] = st.m;
            e.red[kT / 64 + (t >> 6)] = st.s;
        }
        __syncthreads();
        st = {e.red[0], e.red[kT / 64]};
#pragma unroll
        for (int w = 1; w < kT / 64; ++w) st = join(st, {e.red[w], e.red[kT / 64 + w]}, c);
        m = st.m;
        log2s = log2f(st.s);
        lse = st.s > 0.0f ? m * inv_tau + logf(st.s) : __builtin_nanf("");
        if (e.bad) lse = __builtin_nanf("");
        // the loss, one entry per thread
        float term = 0.0f;
        if (have && p > 0.0f) term = p * ((tl - tmax - logf(psum)) - (e.x[t] * inv_tau - lse));
        const float kl = block_add(term, e.red);
        if (t == 0) {
            if (a.lse) a.lse[row] = lse;
            if (a.loss)
                a.loss[row] = lse != lse ? lse : empty ? 0.0f : weight * a.tau * a.tau * kl;
        }
    } else {
        lse = a.lse_in[row];
        if (e.bad) lse = __builtin_nanf("");
    }
    if (MODE == kDistillForward) return;

    const float S = a.ctl ? a.ctl->scale : a.S;
    float coef = S * weight * a.tau;
    if (empty) coef = 0.0f;
    // q_v from the maximum and the sum, or from lse alone: the difference
    // first, so that large logits do not overflow on their way
    auto prob = [&](float v) {
        if (MODE == kDistillBackward)
            return exp2_fast(__builtin_fmaf(v, inv_tau, -lse) * kLog2e);
        return exp2_fast(__builtin_fmaf(v - m, c, -log2s));
    };
    if (lse != lse) coef = lse;
    __syncthreads();
    for (int v = 8 * t; v < vocab; v += 8 * kT) {
        const Raw8<B> r = load8<B>(x, v, vocab - v);
        float f[8];
        widen8<B>(r, bf16, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float q = prob(f[k]);
            f[k] = empty && coef == 0.0f ? 0.0f : coef * q;
        }
        store8(g, v, vocab - v, a.dtype, f);
    }
    __syncthreads();
    if (t < a.top && idx >= 0 && !empty) {
        float taken = 0.0f;
        for (int j = 0; j < a.top; ++j)
            if (e.idx[j] == idx) taken += e.p[j];
        const float q = prob(e.x[t]);
        store1(g, idx, a.dtype, coef * (q - taken));
    }
}

template <DistillMode MODE>
void distill_mode(const DistillArgs& a, hipStream_t stream) {
    const dim3 grid(static_cast<uint32_t>(a.rows));
    if (a.dtype == ZERO_F32) distill_kernel<4, MODE><<<grid, kT, 0, stream>>>(a);
    else distill_kernel<2, MODE><<<grid, kT, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_distill(const DistillArgs& a, DistillMode mode, hipStream_t stream) {
    if (mode == kDistillForward) distill_mode<kDistillForward>(a, stream);
    else if (mode == kDistillBackward) distill_mode<kDistillBackward>(a, stream);
    else distill_mode<kDistillBoth>(a, stream);
    return hipGetLastError();
}

}  // namespace zero
