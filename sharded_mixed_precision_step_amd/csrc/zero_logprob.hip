// Log probabilities of given tokens, entropy and top alternatives, and their
// gradient.
//
// Forward: one workgroup per row, which goes by once for the running maximum m,
// the sum s of e = 2^d and the sum w of e d, d = (z - m) log2(e) / temperature:
//   lse = m / temperature + ln s,   entropy = ln s - ln 2 * w / s
// For the alternatives each lane also keeps its own largest logit.  The top-th
// largest of 256 groups of lanes' maxima is at most the row's top-th largest
// logit, and few others reach it: a second pass over the row (from registers up
// to 32,768 elements, else mostly from the caches) collects those, and counting
// how many come before each, by value and place, orders them.  A row with too many
// such logits (long ties) has its border found by bisection.
#include "zero_device.h"
#include "zero_model_internal.h"

namespace zero {
namespace {

using namespace dev;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kLowest = -3.402823466e38f;
constexpr float kFar = -200.0f;  // 2^-200 is 0 in fp32

// 2^x by the hardware's instruction: one step off at most
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

struct Stat {
    float m, s, w;  // running maximum, sum of e, sum of e d
};

__device__ __forceinline__ void rescale(Stat& st, float m, float c) {
    const float d = fmaxf((st.m - m) * c, kFar), r = exp2_fast(d);
    st.w = r * __builtin_fmaf(st.s, d, st.w);
    st.s *= r;
    st.m = m;
}

__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
    const float m = fmaxf(a.m, b.m);
    rescale(a, m, c);
    rescale(b, m, c);
    return {m, a.s + b.s, a.w + b.w};
}

template <int N>
__device__ __forceinline__ Stat lanes_join(Stat st, float c) {
#pragma unroll
    for (int d = 1; d < N; d *= 2)
        st = join(st, {__shfl_xor(st.m, d), __shfl_xor(st.s, d), __shfl_xor(st.w, d)}, c);
    return st;
}

template <int B>
__device__ __forceinline__ Raw8<B> load_aligned(const char* at) {
    Raw8<B> r;
#pragma unroll
    for (int k = 0; k < B / 2; ++k) r.v[k] = reinterpret_cast<const u32x4*>(at)[k];
    return r;
}

// One logit whose maximum st.m already has.  A NaN or a difference of NaN makes s
// NaN; d of -inf adds nothing.
__device__ __forceinline__ void add(float& s, float& w, float v, float m, float c) {
    const float d = (v - m) * c, e = exp2_fast(d);
    s += e;
    w = __builtin_fmaf(e, fmaxf(d, kFar), w);
}

// N packs: one maximum and one rescaling for them all.
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
    rescale(st, m, c);
#pragma unroll
    for (int u = 0; u < N; ++u) {
        float s = 0.0f, w = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) add(s, w, f[u][k], m, c);
        st.s += s;
        st.w += w;
    }
}

// Whole numbers in the order of fp32's values, both zeros alike; 0 is below all.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = as_bits(v == 0.0f ? 0.0f : v);
    return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
    return as_float(key ^ (key >> 31 ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t kNoKey = 0x007fffffu;  // -inf's: no alternative

constexpr int kGroups = 256;     // lane groups with a maximum each
constexpr int kCandidates = 512;

// The largest key that at least n of 256 values (four a lane, the same in each
// wave) reach; 0 if there is none but 0.
__device__ __forceinline__ uint32_t nth_largest(const uint32_t (&v)[4], int n) {
    uint32_t key = 0;
    for (int b = 31; b >= 0; --b) {
        const uint32_t up = key | 1u << b;
        int count = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) count += __popcll(__ballot(v[k] >= up));
        if (count >= n) key = up;
    }
    return key;
}

struct Row {
    const char* x;
    const char* body;   // at a 16-byte border
    int head, packs, vocab, edge;
    float edge_x;
};

// Calls f(value, place) for each of the lane's logits.
template <int B, int T, int R, class F>
__device__ __forceinline__ void for_each(const Row& row, const Raw8<B>* held, bool bf16, F f) {
    auto pack = [&](const Raw8<B>& r, int p) {
        float v[8];
        widen8<B>(r, bf16, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) f(v[k], row.head + 8 * p + k);
    };
    if constexpr (R > 0) {
#pragma unroll
        for (int u = 0; u < R; ++u)
            if (static_cast<int>(threadIdx.x) + u * T < row.packs) pack(held[u], threadIdx.x + u * T);
    } else {
        for (int p = threadIdx.x; p < row.packs; p += T)
            pack(load_aligned<B>(row.body + static_cast<int64_t>(p) * 8 * B), p);
    }
    if (row.edge >= 0) f(row.edge_x, row.edge);
}

// T lanes per row; R > 0: the row's body is at most R * T packs, and stays in
// registers.
template <int DT, int T, int R, bool TOP>
__global__ __launch_bounds__(T, 4) void logprob_kernel(const LogprobArgs a, int64_t first) {
    constexpr int B = DT == ZERO_F32 ? 4 : 2;
    constexpr bool bf16 = DT == ZERO_BF16, kHeld = R > 0;
    constexpr int kWaves = T / 64;
    __shared__ Stat row_part[kWaves];
    __shared__ uint32_t group_max[TOP ? kGroups : 1];
    __shared__ uint32_t cand_key[TOP ? kCandidates : 1], cand_at[TOP ? kCandidates : 1];
    __shared__ uint32_t count;
    __shared__ uint32_t counts[2][kWaves];
    const int t = threadIdx.x, wave = t / 64;
    const int64_t row_at = first + blockIdx.x;
    const int64_t id = !a.ids ? 0
                       : a.id_bytes == 8 ? static_cast<const int64_t*>(a.ids)[row_at]
                                         : static_cast<const int32_t*>(a.ids)[row_at];
    if (id < 0) {
        if (t == 0) {
            if (a.logp) a.logp[row_at] = 0.0f;
            if (a.entropy) a.entropy[row_at] = 0.0f;
            if (a.lse) a.lse[row_at] = 0.0f;
        }
        if (TOP && t < a.top) {
            a.top_index[row_at * a.ld_top + t] = -1;
            store1(a.top_logit, row_at * a.ld_top + t, DT, -__builtin_inff());
        }
        return;
    }
    // The row as a head up to the first 16-byte border, packs of eight, and a
    // tail; head and tail, at most 14 elements, lie one to a lane.
    Row row;
    row.vocab = static_cast<int>(a.vocab);
    row.x = static_cast<const char*>(a.logits) + row_at * a.ld * B;
    row.head = static_cast<int>(-reinterpret_cast<uintptr_t>(row.x) & 15) / B;
    row.head = row.head < row.vocab ? row.head : row.vocab;
    row.packs = (row.vocab - row.head) / 8;
    row.body = row.x + row.head * B;
    const int tail = row.head + 8 * row.packs;
    row.edge = t < row.head ? t : t - row.head < row.vocab - tail ? tail + t - row.head : -1;
    row.edge_x = row.edge >= 0 ? load1(row.x, row.edge, DT) : -__builtin_inff();
    const float at_id = a.logp && id < row.vocab ? load1(row.x, id, DT) : 0.0f;

    Raw8<B> held[kHeld ? R : 1];
    if constexpr (kHeld) {
        // places behind the row read as -inf
        const uint32_t fill = B == 4 ? 0xff800000u : bf16 ? 0xff80ff80u : 0xfc00fc00u;
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if (t + u * T < row.packs) {
                held[u] = load_aligned<B>(row.body + static_cast<int64_t>(t + u * T) * 8 * B);
            } else {
#pragma unroll
                for (int k = 0; k < B / 2; ++k) held[u].v[k] = u32x4{fill, fill, fill, fill};
            }
        }
    }
    const float inv_tau = 1.0f / a.tau, c = kLog2e * inv_tau;
    Stat st = {kLowest, 0.0f, 0.0f};
    float lane_max = -__builtin_inff();
    auto took = [&](const Raw8<B>& r) {
        if constexpr (TOP) {
            float v[8];
            widen8<B>(r, bf16, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) lane_max = fmaxf(lane_max, v[k]);
        }
    };
    if constexpr (kHeld) {
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const Raw8<B> r[1] = {held[u]};
            take(st, r, bf16, c);
            took(r[0]);
            __builtin_amdgcn_sched_barrier(0);
        }
    } else {
        constexpr int kUnroll = 4;
        int p0 = 0;
        for (; p0 + kUnroll * T <= row.packs; p0 += kUnroll * T) {
            Raw8<B> r[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                r[u] = load_aligned<B>(row.body + static_cast<int64_t>(p0 + u * T + t) * 8 * B);
            take(st, r, bf16, c);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) took(r[u]);
        }
        for (int p = p0 + t; p < row.packs; p += T) {
            const Raw8<B> r[1] = {load_aligned<B>(row.body + static_cast<int64_t>(p) * 8 * B)};
            take(st, r, bf16, c);
            took(r[0]);
        }
    }
    if (row.edge >= 0) {
        rescale(st, fmaxf(st.m, row.edge_x), c);
        add(st.s, st.w, row.edge_x, st.m, c);
        lane_max = fmaxf(lane_max, row.edge_x);
    }
    st = lanes_join<64>(st, c);
    if ((t & 63) == 0) row_part[wave] = st;
    if constexpr (TOP) {
        float m = lane_max;
#pragma unroll
        for (int d = 1; d < T / kGroups; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
        const uint32_t key = order_key(m);
        if (t % (T / kGroups) == 0) group_max[t / (T / kGroups)] = key > kNoKey ? key : 0;
        if (t == 0) count = 0;
    }
    __syncthreads();
    st = lanes_join<kWaves>(row_part[t % kWaves], c);
    const bool bad = !(st.s > 0.0f) || id >= row.vocab || !(st.m < __builtin_inff());
    if (t == 0) {
        const float nan = __builtin_nanf(""), log_s = logf(st.s);
        if (a.lse) a.lse[row_at] = bad ? nan : __builtin_fmaf(st.m, inv_tau, log_s);
        if (a.entropy) a.entropy[row_at] = bad ? nan : log_s - kLn2 * (st.w / st.s);
        if (a.logp) a.logp[row_at] = bad ? nan : (at_id - st.m) * inv_tau - log_s;
    }
    if constexpr (TOP) {
        int32_t* index = a.top_index + row_at * a.ld_top;
        const int64_t logit = row_at * a.ld_top;
        if (bad) {
            if (t < a.top) {
                index[t] = 0;
                store1(a.top_logit, logit + t, DT, __builtin_nanf(""));
            }
            return;
        }
        uint32_t v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = group_max[4 * (t & 63) + k];
        uint32_t border = nth_largest(v, a.top);
        border = border > kNoKey ? border : kNoKey + 1;
        auto collect = [&](uint32_t key_from, int at_to) {
            for_each<B, T, R>(row, held, bf16, [&](float f, int at) {
                const uint32_t key = order_key(f);
                if (key > key_from || (key == key_from && at <= at_to)) {
                    const uint32_t n = atomicAdd(&count, 1u);
                    if (n < kCandidates) {
                        cand_key[n] = key;
                        cand_at[n] = static_cast<uint32_t>(at);
                    }
                }
            });
            __syncthreads();
        };
        collect(border, 0x7fffffff);
        if (count > kCandidates) {
            // The border by bisection: the largest key that `top` logits reach,
            // then the place up to which those on it are taken.
            int turn = 0;
            auto reach = [&](uint32_t key_from, int at_to) {
                uint32_t n = 0;
                for_each<B, T, R>(row, held, bf16, [&](float f, int at) {
                    const uint32_t key = order_key(f);
                    n += key > key_from || (key == key_from && at <= at_to);
                });
#pragma unroll
                for (int d = 1; d < 64; d *= 2) n += __shfl_xor(n, d);
                if ((t & 63) == 0) counts[turn][wave] = n;
                __syncthreads();
                n = 0;
                for (int w = 0; w < kWaves; ++w) n += counts[turn][w];
                turn ^= 1;
                return n;
            };
            const uint32_t top = static_cast<uint32_t>(a.top);
            uint32_t lo = border, hi = order_key(st.m);  // lo is reached by `top`
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo + 1) / 2;
                if (reach(mid, 0x7fffffff) >= top) lo = mid;
                else hi = mid - 1;
            }
            int from = 0, to = row.vocab - 1;
            while (from < to) {
                const int mid = from + (to - from) / 2;
                if (reach(lo, mid) >= top) to = mid;
                else from = mid + 1;
            }
            __syncthreads();
            if (t == 0) count = 0;
            __syncthreads();
            collect(lo, from);
        }
        const int n = static_cast<int>(count);
        for (int j = t; j < n; j += T) {
            const uint32_t key = cand_key[j], at = cand_at[j];
            int rank = 0;
            for (int k = 0; k < n; ++k)
                rank += cand_key[k] > key || (cand_key[k] == key && cand_at[k] < at);
            if (rank < a.top) {
                index[rank] = static_cast<int32_t>(at);
                store1(a.top_logit, logit + rank, DT, key_value(key));
            }
        }
        if (t < a.top && t >= n) {
            index[t] = -1;
            store1(a.top_logit, logit + t, DT, -__builtin_inff());
        }
    }
}

template <int DT, bool TOP>
hipError_t logprob_size(const LogprobArgs& a, hipStream_t stream) {
    auto run = [&](auto kernel, uint32_t lanes) {
        return in_launches(a.rows, lanes, [&](int64_t first, uint32_t grid) {
            kernel<<<grid, lanes, 0, stream>>>(a, first);
            return hipGetLastError();
        });
    };
    if (a.vocab <= 256 * 4 * 8) return run(logprob_kernel<DT, 256, 4, TOP>, 256);
    if (a.vocab <= 512 * 4 * 8) return run(logprob_kernel<DT, 512, 4, TOP>, 512);
    if (a.vocab <= 1024 * 4 * 8) return run(logprob_kernel<DT, 1024, 4, TOP>, 1024);
    return run(logprob_kernel<DT, 1024, 0, TOP>, 1024);
}

template <int DT>
hipError_t logprob_type(const LogprobArgs& a, hipStream_t stream) {
    return a.top ? logprob_size<DT, true>(a, stream) : logprob_size<DT, false>(a, stream);
}

// ---- gradient --------------------------------------------------------------

constexpr int kGradLanes = 256, kGradPacks = 4;
constexpr int64_t kGradSlice = int64_t{8} * kGradLanes * kGradPacks;  // logits per workgroup

// p_v and log p_v come from lse, so a row's slices are independent.
template <int DT>
__global__ __launch_bounds__(kGradLanes) void logprob_backward_kernel(const LogprobBackwardArgs a,
                                                                      int64_t first,
                                                                      uint32_t slices) {
    constexpr int B = DT == ZERO_F32 ? 4 : 2;
    const int64_t block = first + blockIdx.x;
    const int64_t row = block / slices;
    const int64_t v0 = (block - row * slices) * kGradSlice + threadIdx.x * 8;
    const int64_t id = !a.ids ? 0
                       : a.id_bytes == 8 ? static_cast<const int64_t*>(a.ids)[row]
                                         : static_cast<const int32_t*>(a.ids)[row];
    const float inv_tau = 1.0f / a.tau, S = a.ctl ? a.ctl->scale : a.S;
    float da = a.dlogp ? a.dlogp[row] : 0.0f, db = a.dentropy ? a.dentropy[row] : 0.0f;
    const bool off = id < 0 || (da == 0.0f && db == 0.0f);
    const float lse = off ? 0.0f : id >= a.vocab ? __builtin_nanf("") : a.lse[row];
    const float entropy = db != 0.0f ? a.entropy[row] : 0.0f;
    da = S * da * inv_tau;
    db = S * db * inv_tau;
    Raw8<B> r[kGradPacks];
    if (!off) {
#pragma unroll
        for (int u = 0; u < kGradPacks; ++u) {
            const int64_t v = v0 + u * kGradLanes * 8, left = a.vocab - v;
            r[u] = load8<B>(a.logits, row * a.ld + v, static_cast<int>(left < 8 ? left : 8));
        }
    }
#pragma unroll
    for (int u = 0; u < kGradPacks; ++u) {
        const int64_t v = v0 + u * kGradLanes * 8, left = a.vocab - v;
        float f[8] = {};
        if (!off) {
            widen8<B>(r[u], DT == ZERO_BF16, f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                // the difference first, so that large logits do not overflow
                const float log_p = __builtin_fmaf(f[k], inv_tau, -lse);
                const float p = exp2_fast(log_p * kLog2e);
                // where p is 0, log p may be -inf
                const float rest = __builtin_fmaf(db, fmaxf(log_p, kFar) + entropy, da);
                f[k] = (v + k == id ? da : 0.0f) - p * rest;
            }
        }
        store8(a.grad, row * a.ld_grad + v, static_cast<int>(left < 8 ? left : 8), DT, f);
    }
}

int64_t grad_slices(int64_t vocab) { return (vocab + kGradSlice - 1) / kGradSlice; }

}  // namespace

hipError_t launch_logprob(const LogprobArgs& a, hipStream_t stream) {
    if (a.dtype == ZERO_F32) return logprob_type<ZERO_F32>(a, stream);
    if (a.dtype == ZERO_F16) return logprob_type<ZERO_F16>(a, stream);
    return logprob_type<ZERO_BF16>(a, stream);
}

int64_t logprob_backward_blocks(int64_t rows, int64_t vocab) { return rows * grad_slices(vocab); }

hipError_t launch_logprob_backward(const LogprobBackwardArgs& a, hipStream_t stream) {
    const uint32_t slices = static_cast<uint32_t>(grad_slices(a.vocab));
    auto run = [&](auto kernel) {
        return in_launches(
            logprob_backward_blocks(a.rows, a.vocab), kGradLanes,
            [&](int64_t first, uint32_t grid) {
                kernel<<<grid, kGradLanes, 0, stream>>>(a, first, slices);
                return hipGetLastError();
            });
    };
    if (a.dtype == ZERO_F32) return run(logprob_backward_kernel<ZERO_F32>);
    if (a.dtype == ZERO_F16) return run(logprob_backward_kernel<ZERO_F16>);
    return run(logprob_backward_kernel<ZERO_BF16>);
}

}  // namespace zero
