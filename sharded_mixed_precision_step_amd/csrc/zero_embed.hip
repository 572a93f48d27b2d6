// Rows of a table by token, and the table's gradient.
//
// Forward: a gather, bound by the latency of id -> row -> store for few tokens (16 of
// 131072 x 4096 fp16 2.3 us each in a graph) and by HBM for many (8192 tokens 19 us).
//
// Backward: the table's zeros are most of the bytes where the table is large (8192 tokens
// of 131072 x 4096 fp16: 1.07 of 1.14 GB); 216 us then, of which they take 160 to 171.
// Added to the table's rows instead, the same tokens take 54 us, in fp32 74.
//
// Backward of more than 512 tokens: they are sorted by their row of the table (a
// stable radix sort of 9 bits a pass, so that equal ids keep the tokens' order), and
// the sorted list is cut into pieces of 16 tokens, or more where there are very many.  A
// workgroup adds up a piece's rows in registers, run by run; a run that lies in one
// piece goes straight to its row of the table, one that crosses into others leaves a
// partial row for each, which a second kernel adds up in order.  So one frequent token
// is the work of many workgroups, and the sums' order depends on the ids alone.
#include "zero_device.h"
#include "zero_model_internal.h"

namespace zero {
namespace {

using namespace dev;

constexpr int kLanes = 256;

__device__ __forceinline__ int64_t load_id(const void* ids, int64_t i, int bytes) {
    return bytes == 8 ? static_cast<const int64_t*>(ids)[i]
                      : static_cast<int64_t>(static_cast<const int32_t*>(ids)[i]);
}

// ---- forward ---------------------------------------------------------------

// 2^shift lanes to a token, U packs of eight columns a lane.
template <int TB, int U>
__global__ __launch_bounds__(kLanes) void embed_kernel(const EmbedArgs a, int64_t first, int shift,
                                                       uint32_t slices) {
    const uint32_t block = static_cast<uint32_t>(first + blockIdx.x);  // all of them fit
    const uint32_t group = block / slices;
    const int64_t token = static_cast<int64_t>(group) * (kLanes >> shift) + (threadIdx.x >> shift);
    if (token >= a.tokens) return;
    const int64_t c0 = (static_cast<int64_t>(block - group * slices) * U << shift |
                        (threadIdx.x & ((1 << shift) - 1))) * 8;
    const int64_t id = load_id(a.ids, token, a.id_bytes);
    const void* table = a.table[a.ctl ? (a.ctl->cur & 1) : 0];
    Raw8<TB> r[U];
    const bool live = id >= 0 && id < a.vocab;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = c0 + (int64_t{8} * u << shift), left = a.cols - c;
        r[u] = load8<TB>(table, id * a.ld_t + c, live ? static_cast<int>(left < 8 ? left : 8) : 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = c0 + (int64_t{8} * u << shift), left = a.cols - c;
        float f[8];
        widen8<TB>(r[u], a.t_dtype == ZERO_BF16, f);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            f[k] = id < a.vocab ? (id < 0 ? 0.0f : f[k] * a.scale) : __builtin_nanf("");
        store8(a.y, token * a.ld_y + c, static_cast<int>(left < 8 ? left : 8), a.y_dtype, f);
    }
}

// ---- sort ------------------------------------------------------------------

constexpr int kDigit = 9, kBins = 1 << kDigit;
// Items of a lane: few, so that there are workgroups for every CU, up to 131,072 tokens
// (65536 of 32000 x 8 fp16 55 us with 16, 43 with 4; 16777216 of 50000 x 8 1.82 ms and
// 2.05, since each workgroup's counts are read again).
__host__ __device__ inline int sort_rounds(int64_t tokens) { return tokens <= 131072 ? 4 : 16; }

// A token's key: its row of the table, or vocab (behind all rows) if it has none.
__device__ __forceinline__ uint32_t sort_key(int64_t id, int64_t vocab) {
    return static_cast<uint32_t>(id < 0 || id > vocab ? vocab : id);
}

struct SortPass {
    const void* ids;            // first pass: the keys come from here
    const uint32_t *keys_in, *order_in;
    uint32_t *keys_out, *order_out, *counts;
    int64_t tokens, vocab;
    int32_t id_bytes, shift;
    bool scanned;               // the counts are sums already
};

// The keys of items i0 + r * STEP, all loads under way at once; past the end the
// last one's.
template <int N, int STEP>
__device__ __forceinline__ void load_keys(const SortPass& a, int64_t i0, uint32_t (&key)[N]) {
    const int64_t last = a.tokens - 1;
    if (a.keys_in) {
#pragma unroll
        for (int r = 0; r < N; ++r) {
            const int64_t i = i0 + r * STEP;
            key[r] = a.keys_in[i < last ? i : last];
        }
    } else if (a.id_bytes == 8) {
        int64_t id[N];
#pragma unroll
        for (int r = 0; r < N; ++r) {
            const int64_t i = i0 + r * STEP;
            id[r] = static_cast<const int64_t*>(a.ids)[i < last ? i : last];
        }
#pragma unroll
        for (int r = 0; r < N; ++r) key[r] = sort_key(id[r], a.vocab);
    } else {
        int32_t id[N];
#pragma unroll
        for (int r = 0; r < N; ++r) {
            const int64_t i = i0 + r * STEP;
            id[r] = static_cast<const int32_t*>(a.ids)[i < last ? i : last];
        }
#pragma unroll
        for (int r = 0; r < N; ++r) key[r] = sort_key(id[r], a.vocab);
    }
}

__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A wave's items r * 64 + lane, r < rounds, of which the first `live` exist: how many
// of its earlier ones have the same digit, in `rank`; and the wave's count of each
// digit.  The lanes of a round that share a digit find each other by their bits in
// `peers`; the first of them counts them all and clears the bits.  `peers` and
// `count` are the wave's own, kBins each, and zero at the start.
template <int N>
__device__ __forceinline__ void rank_items(const uint32_t (&key)[N], int shift, int rounds, int live,
                                           unsigned long long* peers, uint32_t* count,
                                           uint32_t (&rank)[N]) {
    const int lane = threadIdx.x & 63;
    const unsigned long long bit = 1ull << lane;
#pragma unroll
    for (int r = 0; r < N; ++r) {
        if (r >= rounds) continue;
        const uint32_t digit = key[r] >> shift & (kBins - 1);
        const bool in = r * 64 + lane < live;
        if (in) atomicOr(&peers[digit], bit);
        wave_fence();
        const unsigned long long same = peers[digit];
        const uint32_t before = count[digit];
        wave_fence();
        rank[r] = before + __popcll(same & (bit - 1));
        if (in && (same & (bit - 1)) == 0) {
            count[digit] = before + __popcll(same);
            peers[digit] = 0;
        }
        wave_fence();
    }
}

// counts[block][digit]
template <int ROUNDS>
__global__ __launch_bounds__(kLanes) void sort_count_kernel(const SortPass a) {
    __shared__ uint32_t bins[kBins];
    for (int d = threadIdx.x; d < kBins; d += kLanes) bins[d] = 0;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kLanes * ROUNDS) + threadIdx.x;
    uint32_t key[ROUNDS];
    load_keys<ROUNDS, kLanes>(a, i0, key);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r)
        if (i0 + r * kLanes < a.tokens) atomicAdd(&bins[key[r] >> a.shift & (kBins - 1)], 1u);
    __syncthreads();
    for (int d = threadIdx.x; d < kBins; d += kLanes)
        a.counts[static_cast<int64_t>(blockIdx.x) * kBins + d] = bins[d];
}

// Up to this many blocks, each adds up the others' counts by itself.
constexpr uint32_t kUnscanned = 64;

// counts[block][digit] becomes the earlier blocks' count of the digit; behind the last
// block, all blocks' count.  64 digits a workgroup, a range of blocks each wave.
constexpr int kScanWaves = 16;
__global__ __launch_bounds__(64 * kScanWaves) void sort_scan_kernel(uint32_t* counts,
                                                                    uint32_t blocks) {
    __shared__ uint32_t sums[kScanWaves][64];
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const uint32_t per = (blocks + kScanWaves - 1) / kScanWaves;
    const uint32_t b0 = wave * per, b1 = b0 + per < blocks ? b0 + per : blocks;
    uint32_t* own = counts + blockIdx.x * 64 + lane;
    uint32_t sum = 0;
#pragma unroll 16
    for (uint32_t b = b0; b < b1; ++b) sum += own[static_cast<int64_t>(b) * kBins];
    sums[wave][lane] = sum;
    __syncthreads();
    uint32_t at = 0;
    for (uint32_t w = 0; w < wave; ++w) at += sums[w][lane];
    if (wave == kScanWaves - 1) own[static_cast<int64_t>(blocks) * kBins] = at + sum;
#pragma unroll 16
    for (uint32_t b = b0; b < b1; ++b) {
        const uint32_t n = own[static_cast<int64_t>(b) * kBins];
        own[static_cast<int64_t>(b) * kBins] = at;
        at += n;
    }
}

// Places the items behind those of lower digits, of earlier blocks, waves and
// rounds, and of lower lanes.
template <int ROUNDS>
__global__ __launch_bounds__(kLanes) void sort_scatter_kernel(const SortPass a) {
    constexpr int kWaves = kLanes / 64, kPer = kBins / kLanes;  // digits a lane adds up
    __shared__ unsigned long long peers[kWaves][kBins];
    __shared__ uint32_t bins[kWaves][kBins];
    __shared__ uint32_t waves[kWaves];
    const int t = threadIdx.x, wave = t / 64, lane = t % 64;
    for (int d = t; d < kWaves * kBins; d += kLanes) {
        peers[0][d] = 0;
        bins[0][d] = 0;
    }
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kLanes * ROUNDS) + wave * 64 * ROUNDS;
    uint32_t key[ROUNDS], rank[ROUNDS], place[ROUNDS];
    load_keys<ROUNDS, 64>(a, i0 + lane, key);
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int64_t i = i0 + r * 64 + lane;
        place[r] = a.order_in ? a.order_in[i < a.tokens ? i : a.tokens - 1]
                              : static_cast<uint32_t>(i);
    }
    // digits kPer * t ..: all blocks' items, and the earlier blocks'
    uint32_t all[kPer] = {}, before[kPer] = {};
    if (a.scanned) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            before[k] = a.counts[static_cast<int64_t>(blockIdx.x) * kBins + kPer * t + k];
            all[k] = a.counts[static_cast<int64_t>(gridDim.x) * kBins + kPer * t + k];
        }
    } else {
#pragma unroll 8
        for (uint32_t b = 0; b < gridDim.x; ++b) {
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const uint32_t n = a.counts[static_cast<int64_t>(b) * kBins + kPer * t + k];
                all[k] += n;
                before[k] += b < blockIdx.x ? n : 0;
            }
        }
    }
    __syncthreads();
    const int64_t left = a.tokens - i0;
    rank_items(key, a.shift, ROUNDS, static_cast<int>(left < 0 ? 0 : left < 64 * ROUNDS
                                                               ? left : 64 * ROUNDS),
               peers[wave], bins[wave], rank);
    uint32_t total = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) total += all[k];
    uint32_t scan = total;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t v = __shfl_up(scan, d);
        scan += lane >= d ? v : 0;
    }
    if (lane == 63) waves[wave] = scan;
    __syncthreads();
    uint32_t start = scan - total;
    for (int w = 0; w < wave; ++w) start += waves[w];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        uint32_t at = start + before[k];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const uint32_t n = bins[w][kPer * t + k];
            bins[w][kPer * t + k] = at;
            at += n;
        }
        start += all[k];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        if (i0 + r * 64 + lane >= a.tokens) continue;
        const uint32_t at = bins[wave][key[r] >> a.shift & (kBins - 1)] + rank[r];
        a.keys_out[at] = key[r];
        a.order_out[at] = place[r];
    }
}

// ---- rows of zeros, and the sort of few tokens beside them ------------------

constexpr int kStartLanes = 1024, kStartWaves = kStartLanes / 64;
constexpr int kSmallRounds = 16;
constexpr int64_t kSmall = kStartLanes * kSmallRounds;  // tokens that one workgroup may sort

struct Fill {
    void* p;
    int64_t cols, ld;          // in halves, an fp32 column two of them
    uint32_t rows, slices;     // workgroups to a row; to 2^(10 - shift) rows if 1
    int32_t shift;             // 2^shift lanes to a row
};

// One pack of 16 bytes a lane and workgroups in order: HBM takes plain stores best one
// after another (1 GiB 171 us; 178 to 198 with four packs a lane or workgroups that go
// on; 128 MB of fp32 26 us with two packs a lane, 21 with one).
__device__ __forceinline__ void fill_zeros(const Fill& f, int64_t tile) {
    const float zero[8] = {};
    int64_t row = 0, c = tile * (8 * kStartLanes) + threadIdx.x * 8;
    if (f.rows > 1) {
        const uint32_t t = static_cast<uint32_t>(tile), group = t / f.slices;
        row = static_cast<int64_t>(group) * (kStartLanes >> f.shift) + (threadIdx.x >> f.shift);
        c = (static_cast<int64_t>(t - group * f.slices) << f.shift |
             (threadIdx.x & ((1 << f.shift) - 1))) * 8;
        if (row >= f.rows) return;
    }
    const int64_t left = f.cols - c;
    store8(f.p, row * f.ld + c, static_cast<int>(left < 8 ? left : 8), ZERO_F16, zero);
}

// All passes over up to kSmall tokens by one workgroup, the items in registers
// during a pass and in LDS between passes, where the peers' bits are during one: 15 us
// for 4096 tokens, 20 for 8192, 32 for 16384, behind the zeros where there are enough.
// (By several workgroups, two launches a pass, it takes 13 to 17 us, and nothing else goes
// on meanwhile.)
constexpr int kPeersWords = kStartWaves * kBins * 2, kBinsWords = kStartWaves * kBins;
__host__ __device__ inline int small_words(int rounds) {
    const int items = rounds * kStartLanes * 6 / 4;
    return (items > kPeersWords ? items : kPeersWords) + kBinsWords;
}
__device__ void sort_small(const SortPass& a, int passes, uint32_t* lds) {
    __shared__ uint32_t waves[kStartWaves];
    const int t = threadIdx.x, wave = t / 64, lane = t % 64;
    const int n = static_cast<int>(a.tokens);
    const int rounds = (n + kStartLanes - 1) / kStartLanes;
    uint32_t* keys = lds;
    uint16_t* places = reinterpret_cast<uint16_t*>(lds + rounds * kStartLanes);
    uint32_t* bins = lds + small_words(rounds) - kBinsWords;  // [wave][digit]
    const int i0 = wave * 64 * rounds + lane, left = n - wave * 64 * rounds;
    uint32_t key[kSmallRounds], at[kSmallRounds];
    uint16_t place[kSmallRounds];
    load_keys<kSmallRounds, 64>(a, i0, key);
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r) place[r] = static_cast<uint16_t>(i0 + r * 64);
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = pass * kDigit;
        for (int d = t; d < kPeersWords / 4; d += kStartLanes)
            reinterpret_cast<u32x4*>(lds)[d] = u32x4{0, 0, 0, 0};
        for (int d = t; d < kBinsWords / 4; d += kStartLanes)
            reinterpret_cast<u32x4*>(bins)[d] = u32x4{0, 0, 0, 0};
        __syncthreads();
        rank_items(key, shift, rounds, left,
                   reinterpret_cast<unsigned long long*>(lds) + wave * kBins, bins + wave * kBins,
                   at);
        __syncthreads();
        {   // thread t: digit t / 2 of eight waves
            constexpr int kHalf = kStartWaves / 2;
            uint32_t* own = bins + (t & 1) * kHalf * kBins + t / 2;
            uint32_t count[kHalf], total = 0;
#pragma unroll
            for (int w = 0; w < kHalf; ++w) {
                count[w] = own[w * kBins];
                total += count[w];
            }
            uint32_t scan = total;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const uint32_t v = __shfl_up(scan, d);
                scan += lane >= d ? v : 0;
            }
            if (lane == 63) waves[wave] = scan;
            __syncthreads();
            uint32_t start = scan - total;
#pragma unroll
            for (int w = 0; w < kStartWaves; ++w) start += w < wave ? waves[w] : 0;
#pragma unroll
            for (int w = 0; w < kHalf; ++w) {
                own[w * kBins] = start;
                start += count[w];
            }
        }
        __syncthreads();
        const bool last = pass == passes - 1;
#pragma unroll
        for (int r = 0; r < kSmallRounds; ++r) {
            if (r >= rounds || i0 + r * 64 >= n) continue;
            at[r] += bins[wave * kBins + (key[r] >> shift & (kBins - 1))];
            if (last) {
                a.keys_out[at[r]] = key[r];
                a.order_out[at[r]] = place[r];
            } else {
                keys[at[r]] = key[r];
                places[at[r]] = place[r];
            }
        }
        if (last) return;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kSmallRounds; ++r) {
            const int i = i0 + r * 64;
            if (r >= rounds || i >= n) continue;
            key[r] = keys[i];
            place[r] = places[i];
        }
        __syncthreads();  // before the peers' bits take their room
    }
}

// Workgroup 0 sorts, if there are passes; the others fill.
__global__ __launch_bounds__(kStartLanes) void embed_start_kernel(const SortPass a, int passes,
                                                                  const Fill f, int64_t first) {
    extern __shared__ __attribute__((aligned(16))) uint32_t sort_lds[];
    const int64_t block = first + blockIdx.x, sorters = passes > 0;
    if (block < sorters) sort_small(a, passes, sort_lds);
    else fill_zeros(f, block - sorters);
}

// ---- sums ------------------------------------------------------------------

constexpr int kPiece = 16;                // sorted tokens whose rows are under way at once

struct Sorted {
    const uint32_t *keys, *order;
    float* parts;                         // [2 * pieces][cols]
    int64_t length;                       // tokens in a piece, a multiple of kPiece
};

// A piece's lanes: 2^shift of them, at least a wave, eight columns each.
struct Lanes {
    int64_t first;
    uint32_t slices;
    int32_t shift;
};
struct PieceAt {
    int64_t piece, c;
    int n;
};
__device__ __forceinline__ PieceAt piece_at(const Lanes& l, int64_t cols) {
    const uint32_t block = static_cast<uint32_t>(l.first + blockIdx.x);  // all of them fit
    const uint32_t group = block / l.slices;
    PieceAt p;
    p.piece = static_cast<int64_t>(group) * (kLanes >> l.shift) +
              __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> l.shift));
    p.c = (static_cast<int64_t>(block - group * l.slices) << l.shift |
           (threadIdx.x & ((1 << l.shift) - 1))) * 8;
    const int64_t left = cols - p.c;
    p.n = static_cast<int>(left < 8 ? left : 8);
    return p;
}

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane));
}

template <int TB>
__device__ __forceinline__ Raw8<TB> old_row(const EmbedBackwardArgs& a, uint32_t row, int64_t c,
                                            int n) {
    return load8<TB>(a.dtable, static_cast<int64_t>(row) * a.ld_dt + c, n);
}
// TB > 0: added to `old`, the row's elements of TB bytes.
template <int TB>
__device__ __forceinline__ void put_row(const EmbedBackwardArgs& a, uint32_t row, int64_t c, int n,
                                        const Raw8<TB == 0 ? 2 : TB>& old, float (&sum)[8]) {
    float f[8] = {};
    if constexpr (TB != 0) widen8<TB>(old, a.dt_dtype == ZERO_BF16, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] = f[k] + sum[k] * a.scale;
    store8(a.dtable, static_cast<int64_t>(row) * a.ld_dt + c, n, a.dt_dtype, sum);
}

// A piece's runs.  A run that came in from the piece before leaves its sum as
// the piece's first partial row, one that only goes on into the next as its
// second.  TB > 0: sums are added to the table's rows, which are loaded with dy's.
// LONG: pieces of more than kPiece tokens.
template <int DB, int TB, bool LONG>
__global__ __launch_bounds__(kLanes) void embed_sum_kernel(const EmbedBackwardArgs a,
                                                           const Sorted s, const Lanes l) {
    const PieceAt p = piece_at(l, a.cols);
    const int64_t length = LONG ? s.length : kPiece, first = p.piece * length;
    // a wave goes as a whole: lanes without columns hold keys that the others read
    if (first >= a.tokens || __ballot(p.n > 0) == 0) return;
    const int64_t end = first + length < a.tokens ? first + length : a.tokens;
    const int lane = threadIdx.x % 64;
    const uint32_t none = static_cast<uint32_t>(a.vocab);
    float sum[8] = {};
    bool came = false;  // the run that is being added up
    for (int64_t i0 = first; i0 < end; i0 += kPiece) {
        const int count = static_cast<int>(end - i0 < kPiece ? end - i0 : kPiece);
        // lane j: the key before the j-th token of these, so that lane count has the
        // last one's and lane count + 1 the one behind; and the j-th token's place
        const int64_t at = i0 - 1 + lane;
        const uint32_t keys = at >= 0 && at < a.tokens && lane < count + 2 ? s.keys[at] : none + 1;
        const uint32_t order = lane < count ? s.order[i0 + lane] : 0;
        uint32_t key = lane_value(keys, 1);
        if (key == none) return;
        if (i0 == first) came = lane_value(keys, 0) == key;
        Raw8<DB> r[kPiece];
        Raw8<TB == 0 ? 2 : TB> old[TB == 0 ? 1 : kPiece];
#pragma unroll
        for (int j = 0; j < kPiece; ++j) {
            const uint32_t own = lane_value(keys, j + 1);
            if (j >= count || own == none) continue;
            r[j] = load8<DB>(a.dy, static_cast<int64_t>(lane_value(order, j)) * a.ld_dy + p.c, p.n);
            if constexpr (TB != 0)
                if (lane_value(keys, j + 2) != own) old[j] = old_row<TB>(a, own, p.c, p.n);
        }
#pragma unroll
        for (int j = 0; j < kPiece; ++j) {
            if (j >= count || key == none) continue;
            float f[8];
            widen8<DB>(r[j], a.dy_dtype == ZERO_BF16, f);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] += f[k];
            const uint32_t next = lane_value(keys, j + 2);
            if (next == key && i0 + j + 1 < end) continue;
            if (came || next == key) {
                store8(s.parts, (2 * p.piece + (came ? 0 : 1)) * a.cols + p.c, p.n, ZERO_F32, sum);
            } else {
                put_row<TB>(a, key, p.c, p.n, old[TB == 0 ? 0 : j], sum);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] = 0.0f;
            came = false;
            key = next;
        }
        if constexpr (!LONG) return;
    }
}

// The runs that go on from the piece in which they began: a wave looks at 512 columns
// of one piece, and adds up the partial rows of up to kShortRun more pieces by itself.
// Of eight neighbouring pieces at most one begins a longer run: the workgroup's waves
// take every kJoinWaves-th of its pieces each, added up in the waves' order.
// (A list of such runs that the sums' kernel makes with an atomic counter costs 9 ns a
// run: 200000 tokens of 50000 x 128 fp16 118 us for the sums, 25 without.)
constexpr int kJoinWaves = 8, kShortRun = 8;
template <int TB>
__global__ __launch_bounds__(64 * kJoinWaves) void embed_join_kernel(const EmbedBackwardArgs a,
                                                                     const Sorted s, int64_t n_first,
                                                                     uint32_t slices) {
    __shared__ float sums[kJoinWaves][64][8];
    __shared__ int64_t long_piece;
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x / 64));
    const uint32_t block = static_cast<uint32_t>(n_first + blockIdx.x);  // all of them fit
    const uint32_t group = block / slices;
    const int64_t piece = static_cast<int64_t>(group) * kJoinWaves + wave;
    const int64_t end = (piece + 1) * s.length;
    const int64_t c = (static_cast<int64_t>(block - group * slices) * 64 + lane) * 8;
    const int64_t left = a.cols - c;
    const int n = static_cast<int>(left < 8 ? left : 8);
    const uint32_t none = static_cast<uint32_t>(a.vocab);
    if (threadIdx.x == 0) long_piece = -1;
    __syncthreads();
    // lane 0: the key before the piece; lane 1: its last one; lane 2 + j: the first one
    // of the j-th piece behind it
    const int64_t at = lane == 0 ? end - s.length - 1 : lane == 1 ? end - 1
                                                                  : end + (lane - 2) * s.length;
    const uint32_t keys = at >= 0 && at < a.tokens ? s.keys[at] : none;
    const uint32_t key = lane_value(keys, 1);
    const uint64_t same = __ballot(keys == key) >> 2;
    if (key != none && (piece == 0 || lane_value(keys, 0) != key) && (same & 1)) {
        const int count = __ffsll(static_cast<long long>(~same)) - 1;
        if (count > kShortRun) {
            if (lane == 0) long_piece = piece;
        } else {
            Raw8<4> r[kShortRun + 1];
            Raw8<TB == 0 ? 2 : TB> old;
            r[0] = load8<4>(s.parts, (2 * piece + 1) * a.cols + c, n);
#pragma unroll
            for (int u = 1; u <= kShortRun; ++u)
                if (u <= count) r[u] = load8<4>(s.parts, 2 * (piece + u) * a.cols + c, n);
            if constexpr (TB != 0) old = old_row<TB>(a, key, c, n);
            float sum[8];
            widen8<4>(r[0], false, sum);
#pragma unroll
            for (int u = 1; u <= kShortRun; ++u) {
                if (u > count) continue;
                float f[8];
                widen8<4>(r[u], false, f);
#pragma unroll
                for (int k = 0; k < 8; ++k) sum[k] += f[k];
            }
            put_row<TB>(a, key, c, n, old, sum);
        }
    }
    __syncthreads();
    const int64_t from = long_piece;
    if (from < 0) return;
    const uint32_t run = s.keys[(from + 1) * s.length];
    float sum[8] = {};
    Raw8<TB == 0 ? 2 : TB> old;
    if (wave == 0) {
        if constexpr (TB != 0) old = old_row<TB>(a, run, c, n);
        widen8<4>(load8<4>(s.parts, (2 * from + 1) * a.cols + c, n), false, sum);
    }
    for (int64_t first = from + 1;; first += 64) {
        // how many of the next 64 pieces the run came into
        const int64_t i = (first + lane) * s.length;
        const uint64_t in = __ballot(i < a.tokens && s.keys[i < a.tokens ? i : 0] == run);
        const int count = ~in ? __ffsll(static_cast<long long>(~in)) - 1 : 64;
        Raw8<4> r[64 / kJoinWaves];
#pragma unroll
        for (int u = 0; u < 64 / kJoinWaves; ++u) {
            const int j = u * kJoinWaves + wave;
            r[u] = load8<4>(s.parts, 2 * (first + j) * a.cols + c, j < count ? n : 0);
        }
#pragma unroll
        for (int u = 0; u < 64 / kJoinWaves; ++u) {
            float f[8];
            widen8<4>(r[u], false, f);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] += f[k];
        }
        if (count < 64) break;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sums[wave][lane][k] = sum[k];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < kJoinWaves; ++w) {
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] += sums[w][lane][k];
    }
    put_row<TB>(a, run, c, n, old, sum);
}

// ---- few tokens ------------------------------------------------------------
// Up to kFew tokens need no sort and one launch.  A wave takes a token and 512
// columns; the lanes compare all ids with its own, which says whether it is the first
// with that id and, if so, which others it adds up, in order.  Other workgroups write
// the zeros, of the rows that no id names.

// (100 tokens of 32000 x 4096 fp16 38 us, 52 by the sort; with up to 1,024 the ids a lane
// holds leave the zeros' workgroups too few waves: 1 GiB 232 us instead of 177.)

constexpr int kFew = 512, kFewKeys = kFew / 64;
constexpr int kFewAtOnce = 8;

struct Few {
    uint32_t sum_blocks, token_slices;  // workgroups that add up; waves to a token
    uint32_t rows, fill_slices;         // of the table; workgroups to a row or rows
    int64_t halves;                     // in a row, an fp32 column two of them
    int32_t shift;                      // 2^shift lanes to a row of zeros
};

template <int DB, int TB>
__device__ __forceinline__ void few_sum(const EmbedBackwardArgs& a, const Few& f, int64_t job) {
    __shared__ uint16_t lists[kLanes / 64][kFew];  // a wave's tokens with its id
    const int lane = threadIdx.x & 63, n_ids = static_cast<int>(a.tokens);
    const int token = static_cast<int>(static_cast<uint32_t>(job) / f.token_slices);
    if (token >= n_ids) return;
    const int64_t slice = static_cast<uint32_t>(job) - static_cast<uint32_t>(token) * f.token_slices;
    const int64_t c = (slice * 64 + lane) * 8, left = a.cols - c;
    const int n = static_cast<int>(left < 8 ? left : 8);
    SortPass p = {};
    p.ids = a.ids;
    p.tokens = a.tokens; p.vocab = a.vocab; p.id_bytes = a.id_bytes;
    uint32_t key[kFewKeys];
    load_keys<kFewKeys, 64>(p, lane, key);
    // the token's own key, then which others share it
    uint32_t own = 0;
#pragma unroll
    for (int k = 0; k < kFewKeys; ++k)
        if (k == token / 64) own = lane_value(key[k], token % 64);
    if (own == static_cast<uint32_t>(a.vocab)) return;
    uint16_t* list = lists[threadIdx.x / 64];
    int count = 0;
    bool first = true;
#pragma unroll
    for (int k = 0; k < kFewKeys; ++k) {
        const uint64_t same = __ballot(key[k] == own && k * 64 + lane < n_ids);
        const uint64_t earlier = k * 64 + 64 <= token ? ~uint64_t{0}
                                 : k * 64 >= token ? 0 : (uint64_t{1} << (token - k * 64)) - 1;
        if (same & earlier) first = false;
        if (same >> lane & 1)
            list[count + __popcll(same & ((uint64_t{1} << lane) - 1))] =
                static_cast<uint16_t>(k * 64 + lane);
        count += __popcll(same);
    }
    if (!first) return;
    wave_fence();
    Raw8<TB == 0 ? 2 : TB> old;
    if constexpr (TB != 0) old = old_row<TB>(a, own, c, n);
    float sum[8] = {};
    for (int i0 = 0; i0 < count; i0 += kFewAtOnce) {
        const uint32_t mine = list[i0 + lane < count ? i0 + lane : i0];
        Raw8<DB> r[kFewAtOnce];
#pragma unroll
        for (int u = 0; u < kFewAtOnce; ++u)
            if (i0 + u < count) r[u] = load8<DB>(a.dy, lane_value(mine, u) * a.ld_dy + c, n);
#pragma unroll
        for (int u = 0; u < kFewAtOnce; ++u) {
            if (i0 + u >= count) continue;
            float x[8];
            widen8<DB>(r[u], a.dy_dtype == ZERO_BF16, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += x[i];
        }
    }
    put_row<TB>(a, own, c, n, old, sum);
}

__device__ __forceinline__ void few_zeros(const EmbedBackwardArgs& a, const Few& f,
                                          uint32_t block) {
    __shared__ uint32_t named[kLanes];
    const uint32_t group = block / f.fill_slices, per = kLanes >> f.shift;
    const int64_t r0 = static_cast<int64_t>(group) * per;
    named[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.tokens; i += kLanes) {
        const int64_t id = load_id(a.ids, i, a.id_bytes);
        if (id >= r0 && id < r0 + per) named[id - r0] = 1;
    }
    __syncthreads();
    const uint32_t r = threadIdx.x >> f.shift;
    const int64_t c = (static_cast<int64_t>(block - group * f.fill_slices) << f.shift |
                       (threadIdx.x & ((1 << f.shift) - 1))) * 8;
    const int64_t left = f.halves - c;
    const int64_t ld = a.dt_dtype == ZERO_F32 ? 2 * a.ld_dt : a.ld_dt;
    const float zero[8] = {};
    if (r0 + r < f.rows && !named[r])
        store8(a.dtable, (r0 + r) * ld + c, static_cast<int>(left < 8 ? left : 8), ZERO_F16, zero);
}

template <int DB, int TB>
__global__ __launch_bounds__(kLanes) void embed_few_kernel(const EmbedBackwardArgs a, const Few f,
                                                           int64_t first) {
    const int64_t block = first + blockIdx.x;
    if (block < f.sum_blocks) {
        few_sum<DB, TB>(a, f, block * (kLanes / 64) +
                                  __builtin_amdgcn_readfirstlane(threadIdx.x / 64));
    } else if constexpr (TB == 0) {
        few_zeros(a, f, static_cast<uint32_t>(block - f.sum_blocks));
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Tokens in a piece: more than 16 where there are waves enough, 32 for each CU, since
// a long run leaves a partial row in each piece (65536 tokens of 32000 x 4096 fp16 26 us
// to join them in pieces of 16, 9 in pieces of 64; 16777216 of 50000 x 8 610 and 40).
int64_t piece_length(int64_t tokens, int64_t cols) {
    int64_t length = kPiece;
    while (length < 16 * kPiece && ceil_div(tokens, 2 * length) * ceil_div(cols, 512) >= 8192)
        length *= 2;
    return length;
}
int64_t pieces(int64_t tokens, int64_t cols) { return ceil_div(tokens, piece_length(tokens, cols)); }
int64_t up16(int64_t n) { return (n + 15) & ~int64_t{15}; }
int piece_shift(int64_t cols) { return cols <= 512 ? 6 : cols <= 1024 ? 7 : 8; }
int64_t piece_slices(int64_t cols) { return ceil_div(cols, int64_t{8} << piece_shift(cols)); }
int64_t join_slices(int64_t cols) { return ceil_div(cols, 512); }
int64_t join_blocks(int64_t tokens, int64_t cols) {
    return ceil_div(pieces(tokens, cols), kJoinWaves) * join_slices(cols);
}

}  // namespace

namespace {

// Lanes per token, as a power of two: what its columns need, up to a workgroup, with
// two packs a lane beyond that (a workgroup per token whatever its width: 32768 tokens x
// 64 fp16 23.8 us, 4.0 so).
int embed_shift(int64_t cols) {
    int shift = 0;
    while (shift < 8 && (int64_t{8} << shift) < cols) ++shift;
    return shift;
}
int64_t embed_slices(int64_t cols) { return cols <= 2048 ? 1 : ceil_div(cols, 4096); }

}  // namespace

int64_t embed_blocks(int64_t tokens, int64_t cols) {
    return ceil_div(tokens, kLanes >> embed_shift(cols)) * embed_slices(cols);
}

hipError_t launch_embed(const EmbedArgs& a, hipStream_t stream) {
    const int shift = embed_shift(a.cols);
    const uint32_t slices = static_cast<uint32_t>(embed_slices(a.cols));
    return in_launches(embed_blocks(a.tokens, a.cols), kLanes, [&](int64_t first, uint32_t grid) {
        auto run = [&](auto kernel) { kernel<<<grid, kLanes, 0, stream>>>(a, first, shift, slices); };
        if (a.t_dtype == ZERO_F32) a.cols <= 2048 ? run(embed_kernel<4, 1>) : run(embed_kernel<4, 2>);
        else a.cols <= 2048 ? run(embed_kernel<2, 1>) : run(embed_kernel<2, 2>);
        return hipGetLastError();
    });
}

EmbedWorkspace embed_workspace(int64_t tokens, int64_t cols) {
    EmbedWorkspace w;
    int64_t at = 0;
    for (int k = 0; k < 2; ++k) {
        w.keys[k] = at;
        at = up16(at + 4 * tokens);
        w.order[k] = at;
        at = up16(at + 4 * tokens);
    }
    w.counts = at;
    at = up16(at + 4 * kBins * (1 + ceil_div(tokens, kLanes * sort_rounds(tokens))));
    w.parts = at;
    w.bytes = at + 4 * 2 * pieces(tokens, cols) * cols;
    return w;
}

namespace {

// The zeros' workgroups, in halves of 16 bits: of a table whose rows leave no gap, of
// one with strided rows.
int64_t halves(int64_t cols, int32_t dtype) { return dtype == ZERO_F32 ? 2 * cols : cols; }
bool gapless(int64_t vocab, int64_t cols, int64_t ld) { return ld == cols || vocab == 1; }
int fill_shift(int64_t cols) {
    int shift = 0;
    while (shift < 10 && (int64_t{8} << shift) < cols) ++shift;
    return shift;
}
int64_t fill_slices(int64_t cols) { return ceil_div(cols, int64_t{8} << fill_shift(cols)); }
int64_t fill_tiles(int64_t vocab, int64_t cols, int64_t ld) {
    if (gapless(vocab, cols, ld)) return ceil_div(vocab * cols, 8 * kStartLanes);
    return ceil_div(vocab, kStartLanes >> fill_shift(cols)) * fill_slices(cols);
}

}  // namespace

namespace {

int few_shift(int64_t cols) {
    int shift = 0;
    while (shift < 8 && (int64_t{8} << shift) < cols) ++shift;
    return shift;
}
int64_t few_sum_blocks(int64_t tokens, int64_t cols) {
    return ceil_div(tokens * ceil_div(cols, 512), kLanes / 64);
}
int64_t few_fill_blocks(int64_t vocab, int64_t cols) {
    return ceil_div(vocab, kLanes >> few_shift(cols)) * ceil_div(cols, int64_t{8} << few_shift(cols));
}
bool is_few(int64_t tokens, int64_t vocab, int64_t cols, int32_t dt_dtype) {
    return tokens > 0 && tokens <= kFew &&
           few_sum_blocks(tokens, cols) + few_fill_blocks(vocab, halves(cols, dt_dtype)) <= 0x7fffffff;
}

}  // namespace

int64_t embed_backward_blocks(int64_t tokens, int64_t vocab, int64_t cols, int64_t ld_dt,
                              int32_t dt_dtype) {
    const int64_t sum = ceil_div(pieces(tokens, cols), kLanes >> piece_shift(cols)) * piece_slices(cols);
    const int64_t fill = 1 + fill_tiles(vocab, halves(cols, dt_dtype), halves(ld_dt, dt_dtype));
    const int64_t join = join_blocks(tokens, cols);
    return sum > fill ? (sum > join ? sum : join) : (fill > join ? fill : join);
}

namespace {

// The whole sort of many tokens; the last pass's keys and order.
hipError_t sort_many(SortPass p, uint32_t* const (&keys)[2], uint32_t* const (&order)[2],
                     hipStream_t stream, Sorted* s) {
    const int rounds = sort_rounds(p.tokens);
    const uint32_t grid = static_cast<uint32_t>(ceil_div(p.tokens, kLanes * rounds));
    int to = 0;
    p.scanned = grid > kUnscanned;
    for (p.shift = 0; p.vocab >> p.shift; p.shift += kDigit, to ^= 1) {
        p.keys_out = keys[to];
        p.order_out = order[to];
        if (rounds == 4) sort_count_kernel<4><<<grid, kLanes, 0, stream>>>(p);
        else sort_count_kernel<16><<<grid, kLanes, 0, stream>>>(p);
        if (p.scanned)
            sort_scan_kernel<<<kBins / 64, 64 * kScanWaves, 0, stream>>>(p.counts, grid);
        if (rounds == 4) sort_scatter_kernel<4><<<grid, kLanes, 0, stream>>>(p);
        else sort_scatter_kernel<16><<<grid, kLanes, 0, stream>>>(p);
        p.keys_in = keys[to];
        p.order_in = order[to];
    }
    s->keys = p.keys_in;
    s->order = p.order_in;
    return hipGetLastError();
}

// Whether one workgroup sorts beside the zeros, or several in launches of their own.  Beyond
// 8,192 tokens the zeros have to hide what one takes more, 11 KB a token (fp16, by one and
// by several: 16384 of 5000 x 64 46 us and 30, of 32000 x 4096 108 and 120).  Up to that,
// one: 8192 of 131072 x 4096 216 and 231, 4096 of 32000 x 512 31 and 37, 1024 of 1000 x 512
// 21 and 24.  Where no zeros hide it, adding to the table, the two are alike up to 4,096
// tokens (1024 of 1000 x 512 24 and 24, 4096 of 32000 x 512 30 and 30), but at 8,192 one
// is the slower, which this rule does not tell apart (300 x 64 26 and 19, 131072 x 4096 54
// and 48; with the few zeros of 300 x 64 25 and 20, of 1000 x 4096 46 and 42).
bool one_sorts(int64_t tokens, int64_t zeros) {
    return tokens <= 8192 || (tokens <= kSmall && zeros / 11000 >= tokens - 8192);
}

template <int TB>
hipError_t sum_and_join(const EmbedBackwardArgs& a, const Sorted& s, hipStream_t stream) {
    const int shift = piece_shift(a.cols);
    const int64_t slices = piece_slices(a.cols);
    const hipError_t e = in_launches(
        ceil_div(pieces(a.tokens, a.cols), kLanes >> shift) * slices, kLanes,
        [&](int64_t first, uint32_t grid) {
            const Lanes l = {first, static_cast<uint32_t>(slices), shift};
            auto run = [&](auto kernel) { kernel<<<grid, kLanes, 0, stream>>>(a, s, l); };
            const bool is_long = s.length > kPiece;
            if (a.dy_dtype == ZERO_F32)
                is_long ? run(embed_sum_kernel<4, TB, true>) : run(embed_sum_kernel<4, TB, false>);
            else
                is_long ? run(embed_sum_kernel<2, TB, true>) : run(embed_sum_kernel<2, TB, false>);
            return hipGetLastError();
        });
    if (e != hipSuccess || a.tokens <= s.length) return e;
    return in_launches(join_blocks(a.tokens, a.cols), 64 * kJoinWaves,
                       [&](int64_t first, uint32_t grid) {
                           embed_join_kernel<TB><<<grid, 64 * kJoinWaves, 0, stream>>>(
                               a, s, first, static_cast<uint32_t>(join_slices(a.cols)));
                           return hipGetLastError();
                       });
}

template <int TB>
hipError_t launch_few(const EmbedBackwardArgs& a, hipStream_t stream) {
    Few f = {};
    f.sum_blocks = static_cast<uint32_t>(few_sum_blocks(a.tokens, a.cols));
    f.token_slices = static_cast<uint32_t>(ceil_div(a.cols, 512));
    f.rows = static_cast<uint32_t>(a.vocab);
    f.halves = halves(a.cols, a.dt_dtype);
    f.shift = few_shift(f.halves);
    f.fill_slices = static_cast<uint32_t>(ceil_div(f.halves, int64_t{8} << f.shift));
    return in_launches(f.sum_blocks + (TB == 0 ? few_fill_blocks(a.vocab, f.halves) : 0), kLanes,
                       [&](int64_t first, uint32_t grid) {
                           if (a.dy_dtype == ZERO_F32)
                               embed_few_kernel<4, TB><<<grid, kLanes, 0, stream>>>(a, f, first);
                           else embed_few_kernel<2, TB><<<grid, kLanes, 0, stream>>>(a, f, first);
                           return hipGetLastError();
                       });
}

}  // namespace

hipError_t launch_embed_backward(const EmbedBackwardArgs& a, hipStream_t stream) {
    if (is_few(a.tokens, a.vocab, a.cols, a.dt_dtype)) {
        if (!a.accumulate) return launch_few<0>(a, stream);
        return a.dt_dtype == ZERO_F32 ? launch_few<4>(a, stream) : launch_few<2>(a, stream);
    }
    Sorted s = {};
    SortPass p = {};
    int passes = 0;  // of the first launch's own sort
    size_t lds = 0;
    if (a.tokens > 0) {
        const EmbedWorkspace w = embed_workspace(a.tokens, a.cols);
        uint32_t *keys[2], *order[2];
        for (int k = 0; k < 2; ++k) {
            keys[k] = reinterpret_cast<uint32_t*>(a.workspace + w.keys[k]);
            order[k] = reinterpret_cast<uint32_t*>(a.workspace + w.order[k]);
        }
        p.ids = a.ids;
        p.counts = reinterpret_cast<uint32_t*>(a.workspace + w.counts);
        s.length = piece_length(a.tokens, a.cols);
        p.tokens = a.tokens; p.vocab = a.vocab; p.id_bytes = a.id_bytes;
        s.parts = reinterpret_cast<float*>(a.workspace + w.parts);
        if (one_sorts(a.tokens, a.accumulate ? 0 : 2 * a.vocab * halves(a.cols, a.dt_dtype))) {
            while (a.vocab >> (passes * kDigit)) ++passes;
            lds = 4 * static_cast<size_t>(
                          small_words(static_cast<int>(ceil_div(a.tokens, kStartLanes))));
            p.keys_out = keys[0];
            p.order_out = order[0];
            s.keys = keys[0];
            s.order = order[0];
        } else {
            const hipError_t e = sort_many(p, keys, order, stream, &s);
            if (e != hipSuccess) return e;
        }
    }
    int64_t tiles = 0;
    Fill f = {};
    if (!a.accumulate) {
        // rows without a gap between them are one long row
        const bool whole = gapless(a.vocab, a.cols, a.ld_dt);
        const int64_t cols = halves(a.cols, a.dt_dtype);
        f.p = a.dtable;
        f.ld = halves(a.ld_dt, a.dt_dtype);
        f.rows = whole ? 1 : static_cast<uint32_t>(a.vocab);
        f.cols = whole ? a.vocab * cols : cols;
        f.shift = fill_shift(cols);
        f.slices = static_cast<uint32_t>(fill_slices(cols));
        tiles = fill_tiles(a.vocab, cols, f.ld);
    }
    const hipError_t e = in_launches(
        tiles + (passes > 0), kStartLanes, [&](int64_t first, uint32_t grid) {
            embed_start_kernel<<<grid, kStartLanes, lds, stream>>>(p, passes, f, first);
            return hipGetLastError();
        });
    if (e != hipSuccess) return e;
    if (a.tokens == 0) return hipSuccess;
    if (!a.accumulate) return sum_and_join<0>(a, s, stream);
    return a.dt_dtype == ZERO_F32 ? sum_and_join<4>(a, s, stream) : sum_and_join<2>(a, s, stream);
}

}  // namespace zero
