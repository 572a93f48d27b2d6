// Log probabilities of given tokens, entropy and top alternatives, and their
// gradient.
//
// Forward: one workgroup per row, which goes by once for the running maximum m,
// the sum s of e = 2^d and the sum w of e d, d = (z - m) log2(e) / temperature:
//   lse = m / temperature + ln s,   entropy = ln s - ln 2 * w / s
// For the alternatives, each lane's largest logit of the row's first part goes into
// 256 groups' maxima: the top-th largest of these is reached by `top` logits at least,
// and by few others.  Packs of eight whose largest reaches it are noted in LDS as the
// row goes by, so that it is read once; the top-th largest of many such maxima is a
// closer border, and only the packs that reach that one are looked into.  Counting how
// many come before each of their logits, by value and place, orders them.  Where too many
// lie on the border, as in long ties, the row is read again for the exact value of the
// top-th largest, and its ties are taken in the order of their places.
//
// Bound by HBM with many rows: 4096 x 131072 fp16 190 us, 204 to 218 with 64 alternatives
// (5.7 and 4.9 to 5.3 TB/s), the vector units busy in three quarters of the cycles; and by
// the row's chain (load, sums, borders, places) with few: 37 x 32001 bf16 with 20
// alternatives 10 us.
#include "zero_device.h"
#include "zero_model_internal.h"

namespace zero {
namespace {

using namespace dev;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kLowest = -3.402823466e38f;
constexpr float kFar = -200.0f;  // 2^-200 is 0 in fp32

// 2^x by the hardware's instruction: one step off at most, for x as it is rounded, which
// is off by 2^-24 |x| itself
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

// N packs: one rescaling for them all.  Leaves each pack's maximum in `own`.
template <int B, int N>
__device__ __forceinline__ void take(Stat& st, const Raw8<B>* r, bool bf16, float c, float* own) {
    float f[N][8];
    float m = st.m;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        widen8<B>(r[u], bf16, f[u]);
        own[u] = f[u][0];
#pragma unroll
        for (int k = 1; k < 8; ++k) own[u] = fmaxf(own[u], f[u][k]);
        m = fmaxf(m, own[u]);
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
// Low bits of a key that a border leaves out, for fewer steps (with those that fp16 has
// 4096 x 131072 273 us to 260); and those that no value of the type has.
constexpr int kCoarse = 16;
template <int DT>
constexpr int kExact = DT == ZERO_F32 ? 0 : DT == ZERO_F16 ? 13 : 16;

constexpr int kGroups = 256;      // lane groups with a maximum each
constexpr int kWide = 160;        // more packs or logits get a closer border first
constexpr int kCollected = 8 * kWide + 16, kRanked = 256;

// Of the numbers of BITS bits that a wave's lanes hold: the largest that at least `top`
// of them reach; 0 if none but 0 is.
template <int BITS, int N>
__device__ __forceinline__ uint32_t nth_largest(const uint32_t (&v)[N], int top) {
    uint32_t key = 0;
    for (int b = BITS - 1; b >= 0; --b) {
        const uint32_t up = key | 1u << b;
        int count = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            count += __popcll(__ballot(v[i] >= up));
        if (count >= top) key = up;
    }
    return key;
}

struct Row {
    const char* x;
    const char* body;   // at a 16-byte border
    int head, packs, vocab, edge;
    float edge_x;
};

// What the alternatives need in LDS: 29 KB with 2,048 packs, so that five workgroups share
// a CU.
template <int PACKS>
struct Tops {
    static constexpr int kPacks = PACKS;
    uint64_t packs[PACKS];           // the packs noted, as entries of their largest
    uint64_t collected[kCollected];  // their logits that reach the border
    uint64_t ranked[kRanked];        // those that reach a closer one
    float group_max[kGroups];
    float border;
    uint32_t n_packs, n, n_ranked;
    uint32_t reach[2][3][16];
};

// Larger entries come first: a value, then the places left over.
__device__ __forceinline__ uint64_t entry(float v, int place) {
    return static_cast<uint64_t>(order_key(v)) << 32 | (0xffffffffu - static_cast<uint32_t>(place));
}
__device__ __forceinline__ float entry_value(uint64_t e) {
    return key_value(static_cast<uint32_t>(e >> 32));
}
__device__ __forceinline__ int entry_place(uint64_t e) {
    return static_cast<int>(0xffffffffu - static_cast<uint32_t>(e));
}

// Adds to a list in LDS; what does not fit is only counted.
__device__ __forceinline__ void push(uint64_t* list, uint32_t& n, int room, uint64_t e) {
    const uint32_t at = atomicAdd(&n, 1u);
    if (at < static_cast<uint32_t>(room)) list[at] = e;
}

// The lowest value whose key without SHIFT bits is this; the lowest finite one for the
// keys below, since -inf is no alternative.
template <int SHIFT>
__device__ __forceinline__ float border_value(uint32_t key) {
    return key <= 0x007fffffu >> SHIFT ? kLowest : key_value(key << SHIFT);
}

// The value itself, where SHIFT bits are none that a value of the type has: a negative
// one's key ends in ones.
template <int SHIFT>
__device__ __forceinline__ float exact_value(uint32_t key) {
    return key_value(key << SHIFT | (key >> (31 - SHIFT) ? 0u : (1u << SHIFT) - 1));
}

// A border that the row's `top` largest reach, from the lanes' maxima so far.
template <int T, class Tops>
__device__ __forceinline__ float maxima_border(Tops& s, float lane_max, int top) {
    const int t = threadIdx.x;
#pragma unroll
    for (int d = 1; d < T / kGroups; d *= 2) lane_max = fmaxf(lane_max, __shfl_xor(lane_max, d));
    if (t % (T / kGroups) == 0) s.group_max[t / (T / kGroups)] = lane_max;
    __syncthreads();
    if (t < 64) {
        uint32_t v[kGroups / 64];
#pragma unroll
        for (int i = 0; i < kGroups / 64; ++i)
            v[i] = order_key(s.group_max[i * 64 + t]) >> kCoarse;
        const uint32_t key = nth_largest<32 - kCoarse>(v, top);
        if (t == 0) s.border = border_value<kCoarse>(key);
    }
    __syncthreads();
    return s.border;
}

template <int T, class Tops>
__device__ __forceinline__ float first_border(Tops& s, float lane_max, int top) {
    if (threadIdx.x == 0) s.n_packs = s.n = s.n_ranked = 0;
    return maxima_border<T>(s, lane_max, top);
}

// A closer one, from a list's first 64 N entries (`top` at least).
template <int N>
__device__ __forceinline__ float closer(const uint64_t* list, int n, int top) {
    const int t = threadIdx.x;
    uint32_t v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = i * 64 + t;
        const uint32_t key = static_cast<uint32_t>(list[at < n ? at : 0] >> (32 + kCoarse));
        v[i] = at < n ? key : 0;
    }
    return border_value<kCoarse>(nth_largest<32 - kCoarse>(v, top));
}
template <class Tops>
__device__ __forceinline__ float next_border(Tops& s, const uint64_t* list, int n, int top) {
    if (threadIdx.x < 64) {
        const float border = n <= 256 ? closer<4>(list, n, top) : closer<16>(list, n, top);
        if (threadIdx.x == 0) s.border = border;
    }
    __syncthreads();
    return s.border;
}

// One of the three keys that cut lo .. hi into four, none at lo.
__device__ __forceinline__ uint32_t cut(uint32_t lo, uint32_t hi, uint32_t i) {
    const uint64_t at = lo + i * ((static_cast<uint64_t>(hi) - lo + 3) / 4);
    return at < hi ? static_cast<uint32_t>(at) : hi;
}

// The row's `top` largest, from memory, where `border` is known to be reached by them:
// two bits of the top-th largest's key a turn, then the logits above it, then as many of
// those alike as there is room for, in order.
template <int DT, int T, class Tops>
__device__ __forceinline__ int search(Tops& s, const Row& row, int top, float border, float largest) {
    constexpr int B = DT == ZERO_F32 ? 4 : 2, kShift = kExact<DT>, kWaves = T / 64;
    constexpr bool bf16 = DT == ZERO_BF16;
    const int t = threadIdx.x, wave = t / 64, lane = t % 64;
    auto pack = [&](int p, float (&v)[8]) {
        widen8<B>(load_aligned<B>(row.body + static_cast<int64_t>(p) * 8 * B), bf16, v);
    };
    uint32_t lo = order_key(border) >> kShift, hi = order_key(largest) >> kShift;
#pragma unroll 1
    for (int turn = 0; lo < hi; turn ^= 1) {
        float at[3];
        uint32_t reach[3] = {};
#pragma unroll
        for (int i = 0; i < 3; ++i) at[i] = border_value<kShift>(cut(lo, hi, i + 1));
#pragma unroll 1
        for (int p = t; p < row.packs; p += T) {
            float v[8];
            pack(p, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
#pragma unroll
                for (int i = 0; i < 3; ++i) reach[i] += v[k] >= at[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            reach[i] += row.edge_x >= at[i];
#pragma unroll
            for (int d = 1; d < 64; d *= 2) reach[i] += __shfl_xor(reach[i], d);
            if (lane == 0) s.reach[turn][i][wave] = reach[i];
        }
        __syncthreads();
        uint32_t from = lo, to = hi;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            uint32_t all = 0;
            for (int w = 0; w < kWaves; ++w) all += s.reach[turn][i][w];
            const uint32_t key = cut(lo, hi, i + 1);
            if (all >= static_cast<uint32_t>(top)) from = key > from ? key : from;
            else to = key - 1 < to ? key - 1 : to;
        }
        lo = from;
        hi = to;
    }
    const float alike = exact_value<kShift>(lo);
    if (t == 0) s.n_ranked = 0;
    __syncthreads();
#pragma unroll 1
    for (int p = t; p < row.packs; p += T) {
        float v[8];
        pack(p, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (v[k] > alike) push(s.ranked, s.n_ranked, kRanked, entry(v[k], row.head + 8 * p + k));
    }
    if (row.edge_x > alike) push(s.ranked, s.n_ranked, kRanked, entry(row.edge_x, row.edge));
    __syncthreads();
    const int above = static_cast<int>(s.n_ranked), room = top - above;
    const uint64_t below = (uint64_t{1} << lane) - 1;
    // the head and the tail are the first wave's
    const bool edge = row.edge_x == alike, first = row.edge < row.head;
    int taken = 0;
    auto put = [&](int at, int place) {
        if (at < room) s.ranked[above + at] = entry(alike, place);
    };
    const uint64_t heads = __ballot(edge && first), tails = __ballot(edge && !first);
    if (wave == 0) {
        if (edge && first) put(__popcll(heads & below), row.edge);
        if (lane == 0) s.n = __popcll(heads);
    }
    __syncthreads();
    taken = static_cast<int>(s.n);
#pragma unroll 1
    for (int p0 = 0, turn = 0; p0 < row.packs && taken < room; p0 += T, turn ^= 1) {
        float v[8];
        const int p = p0 + t;
        if (p < row.packs) pack(p, v);
        int before = 0, all = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint64_t same = __ballot(p < row.packs && v[k] == alike);
            before += __popcll(same & below);
            all += __popcll(same);
        }
        if (lane == 0) s.reach[turn][0][wave] = static_cast<uint32_t>(all);
        __syncthreads();
        for (int w = 0; w < kWaves; ++w) {
            const int n = static_cast<int>(s.reach[turn][0][w]);
            before += w < wave ? n : 0;
            all = w == 0 ? n : all + n;
        }
        if (p < row.packs) {
            int at = taken + before;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (v[k] == alike) put(at++, row.head + 8 * p + k);
        }
        taken += all;
    }
    if (wave == 0) {
        if (edge && !first) put(taken + __popcll(tails & below), row.edge);
        if (lane == 0) s.n_packs = taken + __popcll(tails);
    }
    __syncthreads();
    taken = static_cast<int>(s.n_packs);
    return above + (taken < room ? taken : room);
}

// The entries among which the row's `top` largest logits are, and how many they are.
// s.packs holds the s.n_packs packs that reach `border`, as far as they fit.
template <int DT, int T, class Tops>
__device__ __forceinline__ const uint64_t* settle(Tops& s, const Row& row, int top, float border,
                                                  float largest, int* count) {
    constexpr int kPacks = Tops::kPacks, B = DT == ZERO_F32 ? 4 : 2;
    constexpr bool bf16 = DT == ZERO_BF16;
    const int t = threadIdx.x;
    int packs = static_cast<int>(s.n_packs);
    if (__builtin_expect(packs > kPacks, 0)) {  // once more, from memory, with the whole row's border
        auto pack_max = [&](int p) {
            float v[8];
            widen8<B>(load_aligned<B>(row.body + static_cast<int64_t>(p) * 8 * B), bf16, v);
#pragma unroll
            for (int k = 1; k < 8; ++k) v[0] = fmaxf(v[0], v[k]);
            return v[0];
        };
        __syncthreads();
        float lane_max = row.edge_x;
#pragma unroll 1
        for (int p = t; p < row.packs; p += T) lane_max = fmaxf(lane_max, pack_max(p));
        border = first_border<T>(s, lane_max, top);
#pragma unroll 1
        for (int p = t; p < row.packs; p += T) {
            const float m = pack_max(p);
            if (m >= border) push(s.packs, s.n_packs, kPacks, entry(m, p));
        }
        __syncthreads();
        packs = static_cast<int>(s.n_packs);
    }
    if (__builtin_expect(packs <= kPacks, 1)) {
        if (packs > kWide) border = next_border(s, s.packs, packs, top);
        for (int j = t; j < packs; j += T) {
            const uint64_t e = s.packs[j];
            if (!(entry_value(e) >= border)) continue;
            const int p = entry_place(e);
            float v[8];
            widen8<B>(load_aligned<B>(row.body + static_cast<int64_t>(p) * 8 * B), bf16, v);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (v[k] >= border)
                    push(s.collected, s.n, kCollected, entry(v[k], row.head + 8 * p + k));
        }
        if (row.edge_x >= border) push(s.collected, s.n, kCollected, entry(row.edge_x, row.edge));
        __syncthreads();
        const int n = static_cast<int>(s.n);
        *count = n;
        if (__builtin_expect(n <= kWide, 1)) return s.collected;
        if (n <= kCollected) {
            border = next_border(s, s.collected, n, top);
            for (int j = t; j < n; j += T) {
                const uint64_t e = s.collected[j];
                if (entry_value(e) >= border) push(s.ranked, s.n_ranked, kRanked, e);
            }
            __syncthreads();
            *count = static_cast<int>(s.n_ranked);
            if (*count <= kRanked) return s.ranked;
        }
    }
    __syncthreads();  // before its counts are cleared
    *count = search<DT, T>(s, row, top, border, largest);
    return s.ranked;
}

// Writes those of n entries that fewer than `top` others come before, in order.
template <int DT, int T>
__device__ __forceinline__ void put_tops(const uint64_t* entries, int n, const LogprobArgs& a,
                                         int64_t row_at) {
    const int t = threadIdx.x & (T - 1);
    const int64_t out = row_at * a.ld_top;
    // 2^split neighbouring lanes share an entry's comparisons, up to 16
    int split = 4;
    while (split > 0 && n << split > T) --split;
    const int part = t & ((1 << split) - 1);
    for (int j0 = 0; j0 < n; j0 += T >> split) {
        const int j = j0 + (t >> split);
        const uint64_t e = entries[j < n ? j : 0];
        int rank = 0;
#pragma unroll 4
        for (int k = part; k < n; k += 1 << split) rank += entries[k] > e;
        for (int d = 1; d < 1 << split; d *= 2) rank += __shfl_xor(rank, d);
        if (j >= n || part != 0 || rank >= a.top) continue;
        a.top_index[out + rank] = entry_place(e);
        store1(a.top_logit, out + rank, DT, entry_value(e));
    }
    for (int j = t; j < a.top; j += T) {
        if (j < n) continue;
        a.top_index[out + j] = -1;
        store1(a.top_logit, out + j, DT, -__builtin_inff());
    }
}

__device__ __forceinline__ int64_t load_id(const void* ids, int64_t row, int bytes) {
    if (!ids) return 0;
    return bytes == 8 ? static_cast<const int64_t*>(ids)[row]
                      : static_cast<int64_t>(static_cast<const int32_t*>(ids)[row]);
}

// A row as a head up to the first 16-byte border, packs of eight, and a tail; head
// and tail, at most 14 elements, lie one to a lane t.
template <int DT>
__device__ __forceinline__ Row row_of(const LogprobArgs& a, int64_t row_at, int t) {
    constexpr int B = DT == ZERO_F32 ? 4 : 2;
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
    return row;
}

// The lane's packs p0 + u * T + t; places behind the row read as -inf.
template <int DT, int T, int R>
__device__ __forceinline__ void load_packs(const Row& row, int p0, int t,
                                           Raw8<DT == ZERO_F32 ? 4 : 2>* r) {
    constexpr int B = DT == ZERO_F32 ? 4 : 2;
    constexpr uint32_t fill = B == 4 ? 0xff800000u : DT == ZERO_BF16 ? 0xff80ff80u : 0xfc00fc00u;
#pragma unroll
    for (int u = 0; u < R; ++u) {
        const int p = p0 + u * T + t;
        if (p < row.packs) {
            r[u] = load_aligned<B>(row.body + static_cast<int64_t>(p) * 8 * B);
        } else {
#pragma unroll
            for (int k = 0; k < B / 2; ++k) r[u].v[k] = u32x4{fill, fill, fill, fill};
        }
    }
}

__device__ __forceinline__ void take_edge(Stat& st, const Row& row, float c) {
    if (row.edge < 0) return;
    rescale(st, fmaxf(st.m, row.edge_x), c);
    add(st.s, st.w, row.edge_x, st.m, c);
}

// The outputs of a row that has no alternatives of its own: left out, or bad.
template <int DT, int T>
__device__ __forceinline__ void put_none(const LogprobArgs& a, int64_t row_at, int t, int32_t at,
                                         float logit) {
    for (int j = t; j < a.top; j += T) {
        a.top_index[row_at * a.ld_top + j] = at;
        store1(a.top_logit, row_at * a.ld_top + j, DT, logit);
    }
}

template <int DT, int T, bool TOP>
__device__ __forceinline__ void put_left_out(const LogprobArgs& a, int64_t row_at, int t) {
    if (t == 0) {
        if (a.logp) a.logp[row_at] = 0.0f;
        if (a.entropy) a.entropy[row_at] = 0.0f;
        if (a.lse) a.lse[row_at] = 0.0f;
    }
    if constexpr (TOP) put_none<DT, T>(a, row_at, t, -1, -__builtin_inff());
}

// The row's numbers from its statistic; whether it is bad.
template <int DT, int T, bool TOP>
__device__ __forceinline__ bool put_row(const LogprobArgs& a, int64_t row_at, int t, const Stat& st,
                                        int64_t id, float at_id, float inv_tau) {
    const bool bad = !(st.s > 0.0f) || id >= a.vocab || !(st.m < __builtin_inff());
    if (t == 0) {
        const float nan = __builtin_nanf(""), log_s = logf(st.s);
        if (a.lse) a.lse[row_at] = bad ? nan : __builtin_fmaf(st.m, inv_tau, log_s);
        if (a.entropy) a.entropy[row_at] = bad ? nan : log_s - kLn2 * (st.w / st.s);
        if (a.logp) a.logp[row_at] = bad ? nan : (at_id - st.m) * inv_tau - log_s;
    }
    if constexpr (TOP) {
        if (bad) put_none<DT, T>(a, row_at, t, 0, __builtin_nanf(""));
    }
    return bad;
}

// ---- a wave per row ----------------------------------------------------------
// Rows of up to 2,048 stay in a wave's registers, four packs a lane, and need no
// barrier.  The top-th largest of the 256 packs' maxima is the border; the logits
// that reach it take their places in LDS by ballots.  65536 x 256 fp16 31 us, 74 with 20
// alternatives (a workgroup per row 196 and 275); 65536 x 2000 56 and 119.

constexpr int kWavePacks = 4, kWaveRows = 4;
constexpr int kWaveEntries = 256;

template <int DT, bool TOP>
__global__ __launch_bounds__(64 * kWaveRows, 8) void logprob_wave_kernel(const LogprobArgs a,
                                                                         int64_t first) {
    constexpr int B = DT == ZERO_F32 ? 4 : 2, R = kWavePacks;
    constexpr bool bf16 = DT == ZERO_BF16;
    __shared__ uint64_t lists[TOP ? kWaveRows : 1][TOP ? kWaveEntries : 1];
    const int t = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int64_t row_at = (first + blockIdx.x) * kWaveRows + wave;
    if (row_at >= a.rows) return;
    const int64_t id = load_id(a.ids, row_at, a.id_bytes);
    if (id < 0) {
        put_left_out<DT, 64, TOP>(a, row_at, t);
        return;
    }
    const Row row = row_of<DT>(a, row_at, t);
    const float at_id = a.logp && id < row.vocab ? load1(row.x, id, DT) : 0.0f;
    Raw8<B> r[R];
    load_packs<DT, 64, R>(row, 0, t, r);
    const float inv_tau = 1.0f / a.tau, c = kLog2e * inv_tau;
    Stat st = {kLowest, 0.0f, 0.0f};
    float own[R];
#pragma unroll
    for (int u = 0; u < R; ++u)
        if (u * 64 < row.packs) take<B, 1>(st, r + u, bf16, c, own + u);
        else own[u] = -__builtin_inff();
    take_edge(st, row, c);
    st = lanes_join<64>(st, c);
    const bool bad = put_row<DT, 64, TOP>(a, row_at, t, st, id, at_id, inv_tau);
    if constexpr (TOP) {
        if (bad) return;
        uint32_t v[R];
#pragma unroll
        for (int u = 0; u < R; ++u) v[u] = order_key(own[u]) >> kCoarse;
        const float border = border_value<kCoarse>(nth_largest<32 - kCoarse>(v, a.top));
        const uint64_t below = (uint64_t{1} << t) - 1;
        // f(value, place) for each logit of the wave's packs that reach the border, and
        // of its edges, by whole waves
        auto each = [&](auto f) {
#pragma unroll
            for (int u = 0; u < R; ++u) {
                if (__ballot(own[u] >= border) == 0) continue;
                float x[8];
                widen8<B>(r[u], bf16, x);
#pragma unroll
                for (int k = 0; k < 8; ++k) f(x[k], row.head + 8 * (u * 64 + t) + k);
            }
            f(row.edge_x, row.edge);
        };
        uint64_t* list = lists[wave];
        int n = 0;
        auto collect = [&](auto wanted) {
            n = 0;
            each([&](float x, int place) {
                const uint64_t in = __ballot(wanted(x));
                const int at = n + __popcll(in & below);
                if ((in >> t & 1) && at < kWaveEntries) list[at] = entry(x, place);
                n += __popcll(in);
            });
        };
        collect([&](float x) { return x >= border; });
        if (n > kWaveEntries) {
            // the exact value of the top-th largest, bit by bit; the logits above it;
            // those alike in order, as many as there is room for
            constexpr int kShift = kExact<DT>;
            uint32_t lo = order_key(border) >> kShift, hi = order_key(st.m) >> kShift;
#pragma unroll 1
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo) / 2 + ((hi - lo) & 1);
                const float at = border_value<kShift>(mid);
                int reach = 0;
                each([&](float x, int) { reach += __popcll(__ballot(x >= at)); });
                if (reach >= a.top) lo = mid;
                else hi = mid - 1;
            }
            const float alike = exact_value<kShift>(lo);
            collect([&](float x) { return x > alike; });
            auto ties = [&](float x, int place, int before) {
                if (x == alike && n + before < a.top) list[n + before] = entry(x, place);
            };
            const uint64_t edges = __ballot(row.edge_x == alike);
            const uint64_t heads = edges & ((uint64_t{1} << row.head) - 1), tails = edges & ~heads;
            if (t < row.head) ties(row.edge_x, row.edge, __popcll(heads & below));
            n += __popcll(heads);
#pragma unroll
            for (int u = 0; u < R; ++u) {
                if (n >= a.top) continue;
                float x[8];
                widen8<B>(r[u], bf16, x);
                int before = 0, all = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint64_t same = __ballot(x[k] == alike);
                    before += __popcll(same & below);
                    all += __popcll(same);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    ties(x[k], row.head + 8 * (u * 64 + t) + k, before);
                    before += x[k] == alike;
                }
                n += all;
            }
            if (t >= row.head) ties(row.edge_x, row.edge, __popcll(tails & below));
            n += __popcll(tails);
            n = n < a.top ? n : a.top;
        }
        // the wave's writes to its list before its reads of it
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        put_tops<DT, 64>(list, n, a, row_at);
    }
}

// ---- a workgroup per row -------------------------------------------------------

// T lanes per row, which take R packs of eight each at a time; without STREAM that is
// the whole row.  Bounded to 64 registers (eight waves a SIMD): a kernel of more scalar
// registers than that allows held one workgroup of 1,024 a CU instead of two.
template <int DT, int T, int R, bool STREAM, bool TOP>
__global__ __launch_bounds__(T, STREAM && TOP && T == 256 ? 5 : 8) void logprob_kernel(const LogprobArgs a, int64_t first) {
    constexpr int B = DT == ZERO_F32 ? 4 : 2;
    constexpr bool bf16 = DT == ZERO_BF16;
    constexpr int kWaves = T / 64;
    // of a row that is held, few more than `top` packs reach the first border
    using Lds = Tops<STREAM ? 2048 : 512>;
    __shared__ Stat row_part[kWaves];
    __shared__ __attribute__((aligned(16))) uint8_t tops[TOP ? sizeof(Lds) : 16];
    Lds& s = *reinterpret_cast<Lds*>(tops);
    const int t = threadIdx.x, wave = t / 64;
    const int64_t row_at = first + blockIdx.x;
    const int64_t id = load_id(a.ids, row_at, a.id_bytes);
    if (id < 0) {
        put_left_out<DT, T, TOP>(a, row_at, t);
        return;
    }
    const Row row = row_of<DT>(a, row_at, t);
    const float at_id = a.logp && id < row.vocab ? load1(row.x, id, DT) : 0.0f;
    float border = 0.0f, lane_max = row.edge_x, own[R];
    auto note = [&](int p0) {
#pragma unroll
        for (int u = 0; u < R; ++u)
            if (own[u] >= border)
                push(s.packs, s.n_packs, Lds::kPacks, entry(own[u], p0 + u * T + t));
    };
    Raw8<B> r[R];
    load_packs<DT, T, R>(row, 0, t, r);
    const float inv_tau = 1.0f / a.tau, c = kLog2e * inv_tau;
    Stat st = {kLowest, 0.0f, 0.0f};
    if constexpr (STREAM) {
        take<B, R>(st, r, bf16, c, own);
    } else {
        // one at a time: its fp32 values have to fit beside the row
#pragma unroll
        for (int u = 0; u < R; ++u) {
            take<B, 1>(st, r + u, bf16, c, own + u);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if constexpr (TOP) {
#pragma unroll
        for (int u = 0; u < R; ++u) lane_max = fmaxf(lane_max, own[u]);
        border = first_border<T>(s, lane_max, a.top);
        note(0);
    }
    if constexpr (STREAM) {
        // The border follows the maxima when four times as much of the row has gone by, so
        // that the list has room for rows of any length.
        int closer_at = 4 * R * T;
        for (int p0 = R * T; p0 < row.packs; p0 += R * T) {
            load_packs<DT, T, R>(row, p0, t, r);
            if (TOP && p0 == closer_at) {
                border = maxima_border<T>(s, lane_max, a.top);
                closer_at *= 4;
            }
            take<B, R>(st, r, bf16, c, own);
            if constexpr (TOP) {
#pragma unroll
                for (int u = 0; u < R; ++u) lane_max = fmaxf(lane_max, own[u]);
                note(p0);
            }
        }
    }
    take_edge(st, row, c);
    st = lanes_join<64>(st, c);
    if ((t & 63) == 0) row_part[wave] = st;
    __syncthreads();
    st = lanes_join<kWaves>(row_part[t % kWaves], c);
    const bool bad = put_row<DT, T, TOP>(a, row_at, t, st, id, at_id, inv_tau);
    if constexpr (TOP) {
        if (bad) return;
        int n;
        const uint64_t* entries = settle<DT, T>(s, row, a.top, border, st.m, &n);
        put_tops<DT, T>(entries, n, a, row_at);
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
    if (a.vocab <= 64 * kWavePacks * 8)
        return in_launches((a.rows + kWaveRows - 1) / kWaveRows, 64 * kWaveRows,
                           [&](int64_t first, uint32_t grid) {
                               logprob_wave_kernel<DT, TOP>
                                   <<<grid, 64 * kWaveRows, 0, stream>>>(a, first);
                               return hipGetLastError();
                           });
    if (a.vocab <= 256 * 4 * 8) return run(logprob_kernel<DT, 256, 4, false, TOP>, 256);
    // Many rows go by in small workgroups, so that others load while one settles its
    // alternatives; few rows have a CU each to themselves.  fp16, with 64 alternatives,
    // by 256, 512 and 1,024 lanes: 4096 x 131072 226, 233 and 266 us, 8192 x 20000 116,
    // 135 and 207, 1024 x 131072 73, 68 and 77, 256 x 131072 46, 36 and 33.  Up to 16,384
    // logits the row could be held by 512 lanes; gone by and held, with 20 alternatives:
    // 8192 x 12000 73 and 88 us, 2048 x 12000 24 and 27.  (With 512 to 2,047 rows held is
    // the faster, which this rule does not tell apart: 1024 x 16384 20 and 16, 512 x 12000
    // 12.1 and 11.1; without alternatives they are alike.)
    if (a.rows >= 2048) return run(logprob_kernel<DT, 256, 4, true, TOP>, 256);
    if (a.rows >= 512) return run(logprob_kernel<DT, 512, 4, true, TOP>, 512);
    if (a.vocab <= 512 * 4 * 8) return run(logprob_kernel<DT, 512, 4, false, TOP>, 512);
    if (a.vocab <= 1024 * 4 * 8) return run(logprob_kernel<DT, 1024, 4, false, TOP>, 1024);
    return run(logprob_kernel<DT, 1024, 4, true, TOP>, 1024);
}

template <int DT>
hipError_t logprob_type(const LogprobArgs& a, hipStream_t stream) {
    return a.top ? logprob_size<DT, true>(a, stream) : logprob_size<DT, false>(a, stream);
}

// ---- gradient --------------------------------------------------------------

constexpr int kGradLanes = 256, kGradPacks = 4;

// 2^shift lanes to a row, U packs of eight a lane.  p_v and log p_v come from lse, so
// a row's slices are independent.  Bound by HBM: 2048 x 50001 fp16 74 us, 5.5 TB/s.
template <int DT, int U>
__global__ __launch_bounds__(kGradLanes) void logprob_backward_kernel(const LogprobBackwardArgs a,
                                                                      int64_t first, int shift,
                                                                      uint32_t slices) {
    constexpr int B = DT == ZERO_F32 ? 4 : 2;
    const uint32_t block = static_cast<uint32_t>(first + blockIdx.x);  // all of them fit
    const uint32_t group = block / slices;
    const int64_t row = static_cast<int64_t>(group) * (kGradLanes >> shift) + (threadIdx.x >> shift);
    if (row >= a.rows) return;
    const int64_t v0 = (static_cast<int64_t>(block - group * slices) * U << shift |
                        (threadIdx.x & ((1 << shift) - 1))) * 8;
    const int64_t id = load_id(a.ids, row, a.id_bytes);
    const float inv_tau = 1.0f / a.tau, S = a.ctl ? a.ctl->scale : a.S;
    float da = a.dlogp ? a.dlogp[row] : 0.0f, db = a.dentropy ? a.dentropy[row] : 0.0f;
    const bool off = id < 0 || (da == 0.0f && db == 0.0f);
    const float lse = off ? 0.0f : id >= a.vocab ? __builtin_nanf("") : a.lse[row];
    const float entropy = db != 0.0f ? a.entropy[row] : 0.0f;
    da = S * da * inv_tau;
    db = S * db * inv_tau;
    Raw8<B> r[U];
    if (!off) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t v = v0 + (int64_t{8} * u << shift), left = a.vocab - v;
            r[u] = load8<B>(a.logits, row * a.ld + v, static_cast<int>(left < 8 ? left : 8));
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t v = v0 + (int64_t{8} * u << shift), left = a.vocab - v;
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

// Lanes per row, as a power of two: what its packs need, up to a workgroup (a workgroup
// whatever the row: 65536 x 256 fp16 190 us, 15 so), with four packs a lane beyond that.
int grad_shift(int64_t vocab) {
    int shift = 0;
    while (shift < 8 && (int64_t{8} << shift) < vocab) ++shift;
    return shift;
}
bool grad_wide(int64_t vocab) { return vocab > 8 * kGradLanes; }
int64_t grad_slices(int64_t vocab) {
    const int64_t span = 8 * kGradLanes * kGradPacks;
    return grad_wide(vocab) ? (vocab + span - 1) / span : 1;
}

}  // namespace

hipError_t launch_logprob(const LogprobArgs& a, hipStream_t stream) {
    if (a.dtype == ZERO_F32) return logprob_type<ZERO_F32>(a, stream);
    if (a.dtype == ZERO_F16) return logprob_type<ZERO_F16>(a, stream);
    return logprob_type<ZERO_BF16>(a, stream);
}

int64_t logprob_backward_blocks(int64_t rows, int64_t vocab) {
    const int64_t per = kGradLanes >> grad_shift(vocab);
    return (rows + per - 1) / per * grad_slices(vocab);
}

hipError_t launch_logprob_backward(const LogprobBackwardArgs& a, hipStream_t stream) {
    const int shift = grad_shift(a.vocab);
    const uint32_t slices = static_cast<uint32_t>(grad_slices(a.vocab));
    auto run = [&](auto kernel) {
        return in_launches(
            logprob_backward_blocks(a.rows, a.vocab), kGradLanes,
            [&](int64_t first, uint32_t grid) {
                kernel<<<grid, kGradLanes, 0, stream>>>(a, first, shift, slices);
                return hipGetLastError();
            });
    };
    if (grad_wide(a.vocab)) {
        if (a.dtype == ZERO_F32) return run(logprob_backward_kernel<ZERO_F32, kGradPacks>);
        if (a.dtype == ZERO_F16) return run(logprob_backward_kernel<ZERO_F16, kGradPacks>);
        return run(logprob_backward_kernel<ZERO_BF16, kGradPacks>);
    }
    if (a.dtype == ZERO_F32) return run(logprob_backward_kernel<ZERO_F32, 1>);
    if (a.dtype == ZERO_F16) return run(logprob_backward_kernel<ZERO_F16, 1>);
    return run(logprob_backward_kernel<ZERO_BF16, 1>);
}

}  // namespace zero
