// Rows of a table by token, and the table's gradient.
//
// Forward: a gather, bound by the latency of id -> row -> store for few tokens
// and by HBM for many.
//
// Backward: the tokens are sorted by their row of the table (a stable radix sort
// of 6 bits a pass, so that equal ids keep the tokens' order), and the sorted
// list is cut into pieces of 32 tokens.  A workgroup adds up a piece's rows in
// registers, run by run; a run that lies in one piece goes straight to its row
// of the table, one that crosses into others leaves a partial row for each, which
// a second kernel adds up in order.  So one frequent token is the work of many
// workgroups, and the sums' order depends on the ids alone.
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

__device__ __forceinline__ void load_row8(const void* p, int64_t i, int n, int dtype,
                                          float (&f)[8]) {
    if (dtype == ZERO_F32) widen8<4>(load8<4>(p, i, n), false, f);
    else widen8<2>(load8<2>(p, i, n), dtype == ZERO_BF16, f);
}

// ---- forward ---------------------------------------------------------------

constexpr int kSlice = 2 * kLanes * 8;  // columns per workgroup, two packs a lane

template <int TB>
__global__ __launch_bounds__(kLanes) void embed_kernel(const EmbedArgs a, int64_t first,
                                                       uint32_t slices) {
    const int64_t block = first + blockIdx.x;
    const int64_t token = block / slices;
    const int64_t c0 = (block - token * slices) * kSlice + threadIdx.x * 8;
    const int64_t id = load_id(a.ids, token, a.id_bytes);
    const void* table = a.table[a.ctl ? (a.ctl->cur & 1) : 0];
    Raw8<TB> r[2];
    const bool live = id >= 0 && id < a.vocab;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int64_t c = c0 + u * kLanes * 8;
        const int64_t left = a.cols - c;
        r[u] = load8<TB>(table, id * a.ld_t + c, live ? static_cast<int>(left < 8 ? left : 8) : 0);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int64_t c = c0 + u * kLanes * 8;
        const int64_t left = a.cols - c;
        float f[8];
        widen8<TB>(r[u], a.t_dtype == ZERO_BF16, f);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            f[k] = id < a.vocab ? (id < 0 ? 0.0f : f[k] * a.scale) : __builtin_nanf("");
        store8(a.y, token * a.ld_y + c, static_cast<int>(left < 8 ? left : 8), a.y_dtype, f);
    }
}

// ---- sort ------------------------------------------------------------------

constexpr int kDigit = 6, kBins = 1 << kDigit;
constexpr int kSortRounds = 16;
constexpr int kSortItems = kLanes * kSortRounds;  // items per workgroup

// A token's key: its row of the table, or vocab (behind all rows) if it has none.
__device__ __forceinline__ uint32_t sort_key(const void* ids, int64_t i, int bytes,
                                             int64_t vocab) {
    const int64_t id = load_id(ids, i, bytes);
    return static_cast<uint32_t>(id < 0 || id > vocab ? vocab : id);
}

struct SortPass {
    const void* ids;            // first pass: the keys come from here
    const uint32_t *keys_in, *order_in;
    uint32_t *keys_out, *order_out, *counts;
    int64_t tokens, vocab;
    int32_t id_bytes, shift;
};

__device__ __forceinline__ uint32_t pass_key(const SortPass& a, int64_t i) {
    return a.keys_in ? a.keys_in[i] : sort_key(a.ids, i, a.id_bytes, a.vocab);
}

// counts[block][digit]
__global__ __launch_bounds__(kLanes) void sort_count_kernel(const SortPass a) {
    __shared__ uint32_t bins[kBins];
    if (threadIdx.x < kBins) bins[threadIdx.x] = 0;
    __syncthreads();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kSortItems;
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const int64_t i = i0 + r * kLanes + threadIdx.x;
        if (i < a.tokens) atomicAdd(&bins[pass_key(a, i) >> a.shift & (kBins - 1)], 1u);
    }
    __syncthreads();
    if (threadIdx.x < kBins) a.counts[blockIdx.x * kBins + threadIdx.x] = bins[threadIdx.x];
}

// Places the items behind those of lower digits, of earlier blocks, waves and
// rounds, and of lower lanes.
__global__ __launch_bounds__(kLanes) void sort_scatter_kernel(const SortPass a) {
    constexpr int kWaves = kLanes / 64;
    __shared__ uint32_t bins[kWaves][kBins];    // items of a wave so far
    __shared__ uint32_t sums[2][kWaves][kBins]; // all blocks' and earlier blocks' items
    __shared__ uint32_t base[kWaves][kBins];
    const int t = threadIdx.x, wave = t / 64, lane = t % 64;
    bins[wave][lane] = 0;
    uint32_t all = 0, before = 0;
    for (uint32_t b = wave; b < gridDim.x; b += kWaves) {
        const uint32_t n = a.counts[b * kBins + lane];
        all += n;
        before += b < blockIdx.x ? n : 0;
    }
    sums[0][wave][lane] = all;
    sums[1][wave][lane] = before;
    __syncthreads();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kSortItems + wave * 64 * kSortRounds;
    const uint64_t below = (uint64_t{1} << lane) - 1;
    uint32_t key[kSortRounds], rank[kSortRounds];
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const int64_t i = i0 + r * 64 + lane;
        key[r] = i < a.tokens ? pass_key(a, i) : 0;
    }
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const int64_t i = i0 + r * 64 + lane;
        const uint32_t digit = key[r] >> a.shift & (kBins - 1);
        uint64_t peers = __ballot(i < a.tokens);
#pragma unroll
        for (int b = 0; b < kDigit; ++b) {
            const uint64_t set = __ballot(digit >> b & 1);
            peers &= digit >> b & 1 ? set : ~set;
        }
        // the first of them counts them all
        uint32_t old = 0;
        if (i < a.tokens && (peers & below) == 0)
            old = atomicAdd(&bins[wave][digit], static_cast<uint32_t>(__popcll(peers)));
        old = __shfl(old, peers ? __ffsll(static_cast<long long>(peers)) - 1 : lane);
        rank[r] = old + __popcll(peers & below);
    }
    __syncthreads();
    if (wave == 0) {
        uint32_t total = 0, start = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            total += sums[0][w][lane];
            start += sums[1][w][lane];
        }
        uint32_t scan = total;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t v = __shfl_up(scan, d);
            scan += lane >= d ? v : 0;
        }
        start += scan - total;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            base[w][lane] = start;
            start += bins[w][lane];
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const int64_t i = i0 + r * 64 + lane;
        if (i >= a.tokens) continue;
        const uint32_t at = base[wave][key[r] >> a.shift & (kBins - 1)] + rank[r];
        a.keys_out[at] = key[r];
        a.order_out[at] = a.order_in ? a.order_in[i] : static_cast<uint32_t>(i);
    }
}

// ---- sums ------------------------------------------------------------------

constexpr int kPiece = 32;                // sorted tokens per workgroup
constexpr int kSumSlice = kLanes * 8;     // columns per workgroup

struct Sorted {
    const uint32_t *keys, *order;
    float* parts;                         // [2 * pieces][cols]
};

__device__ __forceinline__ void put_row(const EmbedBackwardArgs& a, uint32_t row, int64_t c, int n,
                                        float (&sum)[8]) {
    const int64_t at = static_cast<int64_t>(row) * a.ld_dt + c;
    float old[8] = {};
    if (a.accumulate) load_row8(a.dtable, at, n, a.dt_dtype, old);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] = old[k] + sum[k] * a.scale;
    store8(a.dtable, at, n, a.dt_dtype, sum);
}

// A piece's runs.  A run that came in from the piece before leaves its sum as
// the piece's first partial row, one that only goes on into the next as its
// second.
__global__ __launch_bounds__(kLanes) void embed_sum_kernel(const EmbedBackwardArgs a,
                                                           const Sorted s, int64_t first,
                                                           uint32_t slices) {
    const int64_t block = first + blockIdx.x;
    const int64_t piece = block / slices;
    const int64_t c = (block - piece * slices) * kSumSlice + threadIdx.x * 8;
    if (c >= a.cols) return;
    const int n = static_cast<int>(a.cols - c < 8 ? a.cols - c : 8);
    const int64_t i0 = piece * kPiece;
    const int64_t end = i0 + kPiece < a.tokens ? i0 + kPiece : a.tokens;
    const uint32_t none = static_cast<uint32_t>(a.vocab);
    uint32_t key = s.keys[i0];
    bool came = piece > 0 && s.keys[i0 - 1] == key;
    float sum[8] = {};
    for (int64_t i = i0; i < end && key != none; ++i) {
        float f[8];
        load_row8(a.dy, static_cast<int64_t>(s.order[i]) * a.ld_dy + c, n, a.dy_dtype, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] += f[k];
        const uint32_t next = i + 1 < a.tokens ? s.keys[i + 1] : none + 1;
        if (next == key && i + 1 < end) continue;
        if (came || next == key)
            store8(s.parts, (2 * piece + (came ? 0 : 1)) * a.cols + c, n, ZERO_F32, sum);
        else put_row(a, key, c, n, sum);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] = 0.0f;
        came = false;
        key = next;
    }
}

// The runs that go on from a piece in which they began.
__global__ __launch_bounds__(kLanes) void embed_join_kernel(const EmbedBackwardArgs a,
                                                            const Sorted s, int64_t first,
                                                            uint32_t slices) {
    const int64_t block = first + blockIdx.x;
    const int64_t piece = block / slices;
    const int64_t end = (piece + 1) * kPiece;
    if (end >= a.tokens) return;
    const uint32_t key = s.keys[end];
    const int64_t c = (block - piece * slices) * kSumSlice + threadIdx.x * 8;
    if (key == static_cast<uint32_t>(a.vocab) || s.keys[end - 1] != key || c >= a.cols) return;
    if (piece > 0 && s.keys[end - kPiece] == key && s.keys[end - kPiece - 1] == key) return;
    const int n = static_cast<int>(a.cols - c < 8 ? a.cols - c : 8);
    float sum[8];
    load_row8(s.parts, (2 * piece + 1) * a.cols + c, n, ZERO_F32, sum);
    for (int64_t p = piece + 1; p * kPiece < a.tokens && s.keys[p * kPiece] == key; ++p) {
        float f[8];
        load_row8(s.parts, 2 * p * a.cols + c, n, ZERO_F32, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] += f[k];
    }
    put_row(a, key, c, n, sum);
}

// ---- rows without tokens ---------------------------------------------------

constexpr int kZeroRows = 8;              // rows of the table per workgroup

// The first place of the sorted keys that holds `key` or more.
__device__ __forceinline__ int64_t lower_bound(const uint32_t* keys, int64_t n, uint32_t key) {
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (keys[mid] < key) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kLanes) void embed_zero_kernel(const EmbedBackwardArgs a,
                                                            const Sorted s, int64_t first) {
    __shared__ int64_t at[kZeroRows + 1];
    const int64_t r0 = (first + blockIdx.x) * kZeroRows;
    if (threadIdx.x <= kZeroRows)
        at[threadIdx.x] = a.tokens == 0 ? 0 : lower_bound(s.keys, a.tokens,
                                                          static_cast<uint32_t>(r0 + threadIdx.x));
    __syncthreads();
    const float zero[8] = {};
    for (int r = 0; r < kZeroRows && r0 + r < a.vocab; ++r) {
        if (at[r] != at[r + 1]) continue;
        for (int64_t c = threadIdx.x * 8; c < a.cols; c += kLanes * 8)
            store8(a.dtable, (r0 + r) * a.ld_dt + c,
                   static_cast<int>(a.cols - c < 8 ? a.cols - c : 8), a.dt_dtype, zero);
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t pieces(int64_t tokens) { return ceil_div(tokens, kPiece); }
int64_t up16(int64_t n) { return (n + 15) & ~int64_t{15}; }

}  // namespace

int64_t embed_blocks(int64_t tokens, int64_t cols) { return tokens * ceil_div(cols, kSlice); }

hipError_t launch_embed(const EmbedArgs& a, hipStream_t stream) {
    const uint32_t slices = static_cast<uint32_t>(ceil_div(a.cols, kSlice));
    return in_launches(embed_blocks(a.tokens, a.cols), kLanes, [&](int64_t first, uint32_t grid) {
        if (a.t_dtype == ZERO_F32) embed_kernel<4><<<grid, kLanes, 0, stream>>>(a, first, slices);
        else embed_kernel<2><<<grid, kLanes, 0, stream>>>(a, first, slices);
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
    at = up16(at + 4 * kBins * ceil_div(tokens, kSortItems));
    w.parts = at;
    w.bytes = at + 4 * 2 * pieces(tokens) * cols;
    return w;
}

int64_t embed_backward_blocks(int64_t tokens, int64_t vocab, int64_t cols) {
    const int64_t sum = pieces(tokens) * ceil_div(cols, kSumSlice);
    const int64_t zero = ceil_div(vocab, kZeroRows);
    return sum > zero ? sum : zero;
}

hipError_t launch_embed_backward(const EmbedBackwardArgs& a, hipStream_t stream) {
    Sorted s = {};
    if (a.tokens > 0) {
        const EmbedWorkspace w = embed_workspace(a.tokens, a.cols);
        uint32_t *keys[2], *order[2];
        for (int k = 0; k < 2; ++k) {
            keys[k] = reinterpret_cast<uint32_t*>(a.workspace + w.keys[k]);
            order[k] = reinterpret_cast<uint32_t*>(a.workspace + w.order[k]);
        }
        SortPass p = {};
        p.ids = a.ids;
        p.counts = reinterpret_cast<uint32_t*>(a.workspace + w.counts);
        p.tokens = a.tokens; p.vocab = a.vocab; p.id_bytes = a.id_bytes;
        const uint32_t grid = static_cast<uint32_t>(ceil_div(a.tokens, kSortItems));
        int to = 0;
        for (p.shift = 0; a.vocab >> p.shift; p.shift += kDigit, to ^= 1) {
            p.keys_out = keys[to];
            p.order_out = order[to];
            sort_count_kernel<<<grid, kLanes, 0, stream>>>(p);
            sort_scatter_kernel<<<grid, kLanes, 0, stream>>>(p);
            p.keys_in = keys[to];
            p.order_in = order[to];
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        s.keys = p.keys_in;
        s.order = p.order_in;
        s.parts = reinterpret_cast<float*>(a.workspace + w.parts);
        const uint32_t slices = static_cast<uint32_t>(ceil_div(a.cols, kSumSlice));
        for (int join = 0; join < 2; ++join) {
            const hipError_t e = in_launches(
                pieces(a.tokens) * slices, kLanes, [&](int64_t first, uint32_t grid) {
                    if (join) embed_join_kernel<<<grid, kLanes, 0, stream>>>(a, s, first, slices);
                    else embed_sum_kernel<<<grid, kLanes, 0, stream>>>(a, s, first, slices);
                    return hipGetLastError();
                });
            if (e != hipSuccess) return e;
        }
    }
    if (a.accumulate) return hipSuccess;
    return in_launches(ceil_div(a.vocab, kZeroRows), kLanes, [&](int64_t first, uint32_t grid) {
        embed_zero_kernel<<<grid, kLanes, 0, stream>>>(a, s, first);
        return hipGetLastError();
    });
}

}  // namespace zero
