// Distillation from a teacher's top logits: loss and gradient.
//
// One workgroup per row.  The student's row goes by once for the running
// maximum and sum of its softmax (fp32, from a finite start so that a row of
// -inf stays countable) and once more for the gradient.  Rows of up to 32,768
// elements stay in registers in between (16,384 where only the gradient is made,
// 8,192 where only the loss is); longer ones are read twice, the second time mostly
// from the memory-side cache, which the gradient's streaming stores leave to them:
// 4096 x 131072 fp16 takes 463 us, 4.6 TB/s over the logits read once and the
// gradient written once.  With a tenth of the rows of weight 0, 429 us (494 with
// ordinary stores, 524 also with half the loads under way; 751 with the row held in
// 64 registers a lane, where loading, summing and writing do not overlap).  fp32
// logits: 2048 x 50001 203 us, 4.0 TB/s.
//
// The teacher's entries lie one to four per lane; their softmax joins across
// the workgroup together with the row's, behind one barrier.  The gradient is
// first written as coef * q_v for the whole row; behind a second barrier the
// entries' places are written again with their p_j taken off, each computed
// from the logit read before anything was written, so that one rounding is
// made and the gradient may take the logits' place.
#include "zero_device.h"
#include "zero_train_internal.h"

namespace zero {
namespace {

using namespace dev;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;
constexpr int kUnroll = 4;  // packs of eight a lane has under way

// 2^x by the hardware's instruction: one step off at most
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

struct Stat {
    float m, s;  // running maximum, sum of 2^((x - m) c)
};

__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
    const float m = fmaxf(a.m, b.m);
    return {m, a.s * exp2_fast((a.m - m) * c) + b.s * exp2_fast((b.m - m) * c)};
}

// Over each N neighbouring lanes; the same bits on all of them.
template <int N>
__device__ __forceinline__ Stat lanes_join(Stat st, float c) {
#pragma unroll
    for (int d = 1; d < N; d *= 2)
        st = join(st, {__shfl_xor(st.m, d), __shfl_xor(st.s, d)}, c);
    return st;
}

// Pack `at` bytes behind a row's body: the body in scalar registers, so that a
// lane's packs share one offset.
typedef __amdgpu_buffer_rsrc_t Buffer;
template <int B>
__device__ __forceinline__ Raw8<B> load_pack(Buffer body, int lane, int at) {
    Raw8<B> r;
#pragma unroll
    for (int k = 0; k < B / 2; ++k)
        r.v[k] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(body, lane, at + 16 * k, 0));
    return r;
}

template <int B>
__device__ __forceinline__ Raw8<B> load_aligned(const char* at) {
    Raw8<B> r;
#pragma unroll
    for (int k = 0; k < B / 2; ++k) r.v[k] = reinterpret_cast<const u32x4*>(at)[k];
    return r;
}

// N packs into a running statistic: one maximum and one rescaling for them all.
template <int B, int N>
__device__ __forceinline__ void take(Stat& st, const Raw8<B> (&r)[N], bool bf16, float c) {
    float f[N][8];
    float m = st.m;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        widen8<B>(r[u], bf16, f[u]);
#pragma unroll
        for (int k = 0; k < 8; ++k) m = fmaxf(m, f[u][k]);
    }
    st.s *= exp2_fast((st.m - m) * c);
    st.m = m;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += exp2_fast((f[u][k] - m) * c);
        st.s += s;
    }
}

// T lanes per row; R > 0: the row's body is at most R * T packs, and stays in
// registers.
template <int DT, int T, int R, DistillMode MODE>
__global__ __launch_bounds__(T, 4) void distill_kernel(const DistillArgs a, int64_t first) {
    constexpr int B = DT == ZERO_F32 ? 4 : 2;
    constexpr bool bf16 = DT == ZERO_BF16, kHeld = R > 0;
    constexpr int kWaves = T / 64, kEntries = ZERO_DISTILL_MAX_TOP / T;
    __shared__ __attribute__((aligned(16))) int32_t entry_index[ZERO_DISTILL_MAX_TOP];
    __shared__ __attribute__((aligned(16))) float entry_p[ZERO_DISTILL_MAX_TOP];
    __shared__ Stat row_part[kWaves], top_part[kWaves];
    __shared__ float loss_part[kWaves];
    __shared__ int32_t bad_part[kWaves];
    const int t = threadIdx.x, wave = t / 64;
    const int64_t row = first + blockIdx.x;
    const float weight = a.weight ? a.weight[row] : 1.0f;
    const int vocab = static_cast<int>(a.vocab);
    const char* x = static_cast<const char*>(a.logits) + row * a.ld * B;
    char* g = static_cast<char*>(a.grad) + row * a.ld_grad * B;
    // The row as a head up to the first 16-byte border, packs of eight, and a
    // tail; head and tail, at most 14 elements, lie one to a lane.
    int head = static_cast<int>(-reinterpret_cast<uintptr_t>(x) & 15) / B;
    head = head < vocab ? head : vocab;
    const int packs = (vocab - head) / 8, tail = head + 8 * packs;
    const int edge = t < head ? t : t - head < vocab - tail ? tail + t - head : -1;
    // what is known where to find goes first, all of it at once
    int64_t given[kEntries];
    float top[kEntries];
#pragma unroll
    for (int k = 0; k < kEntries; ++k) {
        given[k] = -1;
        top[k] = 0.0f;
        if (t + k * T < a.top) {
            const int64_t at = row * a.ld_top + t + k * T;
            given[k] = a.index_bytes == 8 ? static_cast<const int64_t*>(a.index)[at]
                                          : static_cast<const int32_t*>(a.index)[at];
            top[k] = load1(a.top_logit, at, a.top_dtype);
        }
    }
    const char* body = x + head * B;
    const float edge_x = edge >= 0 ? load1(x, edge, DT) : -__builtin_inff();

    Raw8<B> held[kHeld ? R : 1];
    if constexpr (kHeld) {
        // places behind the row read as -inf
        constexpr uint32_t kInf32 = 0xff800000u;
        const uint32_t fill = B == 4 ? kInf32 : bf16 ? 0xff80ff80u : 0xfc00fc00u;
        const Buffer buffer =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(body), 0, -1, 0x00020000);
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if ((u + 1) * T <= packs || t + u * T < packs) {
                held[u] = load_pack<B>(buffer, t * 8 * B, u * T * 8 * B);
            } else {
#pragma unroll
                for (int k = 0; k < B / 2; ++k) held[u].v[k] = u32x4{fill, fill, fill, fill};
            }
        }
    }

    if (weight == 0.0f) {
        if (MODE != kDistillBackward && t == 0) {
            if (a.loss) a.loss[row] = 0.0f;
            if (a.lse) a.lse[row] = 0.0f;
        }
        if (MODE != kDistillForward) {
            const float zero[8] = {};
            for (int64_t v = 8 * t; v < vocab; v += 8 * T)
                store8(g, v, static_cast<int>(vocab - v), DT, zero);
        }
        return;
    }

    // the teacher's entries; divided by the temperature as differences only, so
    // that logits of the type's lowest value stay in range
    const float inv_tau = 1.0f / a.tau, c = kLog2e * inv_tau;
    int32_t index[kEntries];
    float at_index[kEntries];
    bool have[kEntries], bad = false;
    Stat top_stat = {kLowest, 0.0f};
#pragma unroll
    for (int k = 0; k < kEntries; ++k) {
        index[k] = -1;
        at_index[k] = 0.0f;
        have[k] = false;
        const float v = top[k];
        top[k] = kLowest;
        if (given[k] >= vocab) {
            bad = true;
        } else if (given[k] >= 0) {
            index[k] = static_cast<int32_t>(given[k]);
            at_index[k] = load1(x, given[k], DT);
            if (!(v < __builtin_inff())) bad = true;  // NaN or +inf
            else if (v > -__builtin_inff()) {
                have[k] = true;
                top[k] = v;
            }
        }
        if (have[k]) top_stat = join(top_stat, {top[k], 1.0f}, c);
    }

    // the row's statistic
    Stat st = {kLowest, 0.0f};
    if constexpr (MODE != kDistillBackward) {
        if constexpr (kHeld) {
            // one at a time: its fp32 values have to fit beside the row
#pragma unroll
            for (int u = 0; u < R; ++u) {
                const Raw8<B> r[1] = {held[u]};
                take(st, r, bf16, c);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            int p0 = 0;
            for (; p0 + kUnroll * T <= packs; p0 += kUnroll * T) {
                Raw8<B> r[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u)
                    r[u] = load_aligned<B>(body + static_cast<int64_t>(p0 + u * T + t) * 8 * B);
                take(st, r, bf16, c);
            }
            for (int p = p0 + t; p < packs; p += T) {
                const Raw8<B> r[1] = {load_aligned<B>(body + static_cast<int64_t>(p) * 8 * B)};
                take(st, r, bf16, c);
            }
        }
        if (edge >= 0) {
            const float m = fmaxf(st.m, edge_x);
            st.s = st.s * exp2_fast((st.m - m) * c) + exp2_fast((edge_x - m) * c);
            st.m = m;
        }
        st = lanes_join<64>(st, c);
    }
    top_stat = lanes_join<64>(top_stat, c);
    const bool wave_bad = __ballot(bad) != 0;
    if ((t & 63) == 0) {
        if (MODE != kDistillBackward) row_part[wave] = st;
        top_part[wave] = top_stat;
        bad_part[wave] = wave_bad;
    }
    __syncthreads();
    // every wave joins the waves' parts, one to a lane
    const int part = t % kWaves;
    if (MODE != kDistillBackward) st = lanes_join<kWaves>(row_part[part], c);
    top_stat = lanes_join<kWaves>(top_part[part], c);
    bad = __ballot(bad_part[part]) != 0;

    const bool empty = top_stat.s == 0.0f;
    const float inv_top = 1.0f / top_stat.s, log_top = logf(top_stat.s);
    float m = 0.0f, log2s = 0.0f, lse;
    if constexpr (MODE == kDistillBackward) {
        lse = bad ? __builtin_nanf("") : a.lse_in[row];
    } else {
        m = st.m;
        log2s = log2f(st.s);
        const float log_s = logf(st.s);
        lse = st.s > 0.0f && !bad ? m * inv_tau + log_s : __builtin_nanf("");
        float term = 0.0f;
#pragma unroll
        for (int k = 0; k < kEntries; ++k) {
            if (!have[k]) continue;
            const float p = exp2_fast((top[k] - top_stat.m) * c) * inv_top;
            const float log_p = (top[k] - top_stat.m) * inv_tau - log_top;
            const float log_q = (at_index[k] - m) * inv_tau - log_s;
            if (p > 0.0f) term += p * (log_p - log_q);
        }
        term = wave_sum(term);
        if ((t & 63) == 0) loss_part[wave] = term;
    }

    float coef = 0.0f;
    // q_v from the maximum and the sum, or from lse alone: the difference
    // first, so that large logits do not overflow on their way
    auto prob = [&](float v) {
        if (MODE == kDistillBackward) return exp2_fast(__builtin_fmaf(v, inv_tau, -lse) * kLog2e);
        return exp2_fast(__builtin_fmaf(v - m, c, -log2s));
    };
    if constexpr (MODE != kDistillForward) {
        coef = (a.ctl ? a.ctl->scale : a.S) * weight * a.tau;
        if (empty) coef = 0.0f;
        if (lse != lse) coef = lse;
#pragma unroll
        for (int k = 0; k < kEntries; ++k) {
            const int j = t + k * T;
            entry_index[j] = index[k];
            entry_p[j] = have[k] ? exp2_fast((top[k] - top_stat.m) * c) * inv_top : 0.0f;
        }
        char* g_body = g + head * B;
        auto put = [&](const Raw8<B>& r, int p) {
            float f[8];
            widen8<B>(r, bf16, f);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = coef * prob(f[k]);
            store8<true>(g_body, static_cast<int64_t>(p) * 8, 8, DT, f);
        };
        if (empty && coef == 0.0f) {
            const float zero[8] = {};
            for (int64_t v = 8 * t; v < vocab; v += 8 * T)
                store8(g, v, static_cast<int>(vocab - v), DT, zero);
        } else {
            if constexpr (kHeld) {
#pragma unroll
                for (int u = 0; u < R; ++u) {
                    if ((u + 1) * T <= packs || t + u * T < packs) put(held[u], t + u * T);
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                int p0 = 0;
                for (; p0 + kUnroll * T <= packs; p0 += kUnroll * T) {
                    Raw8<B> r[kUnroll];
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u)
                        r[u] = load_aligned<B>(body + static_cast<int64_t>(p0 + u * T + t) * 8 * B);
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u) put(r[u], p0 + u * T + t);
                }
                for (int p = p0 + t; p < packs; p += T)
                    put(load_aligned<B>(body + static_cast<int64_t>(p) * 8 * B), p);
            }
            if (edge >= 0) store1(g, edge, DT, coef * prob(edge_x));
        }
    }
    __syncthreads();
    if (MODE != kDistillBackward && t == 0) {
        float kl = loss_part[0];
        for (int w = 1; w < kWaves; ++w) kl += loss_part[w];
        if (a.lse) a.lse[row] = lse;
        // tau^2 may be below fp32's range where tau * kl is not
        if (a.loss)
            a.loss[row] = lse != lse ? lse : empty ? 0.0f : weight * a.tau * (a.tau * kl);
    }
    if constexpr (MODE != kDistillForward) {
        if (empty) return;
        const int groups = (a.top + 3) / 4;  // behind a.top: index -1
#pragma unroll
        for (int k = 0; k < kEntries; ++k) {
            if (index[k] < 0) continue;
            float taken = 0.0f;
            for (int j = 0; j < groups; ++j) {
                const int4 i4 = reinterpret_cast<const int4*>(entry_index)[j];
                const float4 p4 = reinterpret_cast<const float4*>(entry_p)[j];
                taken += i4.x == index[k] ? p4.x : 0.0f;
                taken += i4.y == index[k] ? p4.y : 0.0f;
                taken += i4.z == index[k] ? p4.z : 0.0f;
                taken += i4.w == index[k] ? p4.w : 0.0f;
            }
            store1(g, index[k], DT, coef * (prob(at_index[k]) - taken));
        }
    }
}

template <int DT, DistillMode MODE>
hipError_t distill_size(const DistillArgs& a, hipStream_t stream) {
    auto run = [&](auto kernel, uint32_t lanes) {
        return in_launches(a.rows, lanes, [&](int64_t first, uint32_t grid) {
            kernel<<<grid, lanes, 0, stream>>>(a, first);
            return hipGetLastError();
        });
    };
    // Lanes per row: 256, else 512, where they hold it (37 rows of 32,001: 9.1 us held
    // by 1,024, 14.7 in two passes; 16384 of 10,000: 168 held by 512, 275 by 1,024;
    // the gradient alone 118, 134 in passes of single packs; the loss alone 116 and
    // 110, where holding gains nothing).  Two passes in one call: 1,024 lanes, so
    // that fewer rows wait in the cache (4096 x 131072: 433 us, 489 with 512); one
    // pass: 512 (2048 x 50001, both calls: 134 us, 174 with 1,024, before streaming
    // stores).
    if (a.vocab <= 256 * kUnroll * 8) return run(distill_kernel<DT, 256, kUnroll, MODE>, 256);
    if constexpr (MODE != kDistillForward) {
        if (a.vocab <= 512 * kUnroll * 8) return run(distill_kernel<DT, 512, kUnroll, MODE>, 512);
    }
    if constexpr (MODE == kDistillBoth) {
        if (a.vocab <= 1024 * kUnroll * 8)
            return run(distill_kernel<DT, 1024, kUnroll, MODE>, 1024);
        return run(distill_kernel<DT, 1024, 0, MODE>, 1024);
    } else {
        return run(distill_kernel<DT, 512, 0, MODE>, 512);
    }
}

template <DistillMode MODE>
hipError_t distill_type(const DistillArgs& a, hipStream_t stream) {
    if (a.dtype == ZERO_F32) return distill_size<ZERO_F32, MODE>(a, stream);
    if (a.dtype == ZERO_F16) return distill_size<ZERO_F16, MODE>(a, stream);
    return distill_size<ZERO_BF16, MODE>(a, stream);
}

}  // namespace

hipError_t launch_distill(const DistillArgs& a, DistillMode mode, hipStream_t stream) {
    if (mode == kDistillForward) return distill_type<kDistillForward>(a, stream);
    if (mode == kDistillBackward) return distill_type<kDistillBackward>(a, stream);
    return distill_type<kDistillBoth>(a, stream);
}

}  // namespace zero
