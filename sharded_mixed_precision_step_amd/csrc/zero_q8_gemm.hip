// The product of two q8 matrices, c = a b^T.
//
// Both operands run along k, so both tiles are staged the same way: 128 bytes
// of k per row and step, straight from HBM into LDS, 16 bytes per lane.  A
// step is one scale block, and the matrix cores apply the scales themselves
// (a power of two per row of each operand), so the inner loop has no other
// arithmetic.  Which k a lane's 32 bytes of a step are is free as long as both
// operands agree, since one scale covers the whole step.
#include "zero_device.h"
#include "zero_train_internal.h"

namespace zero {
namespace {

using namespace dev;

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;  // bytes of k per step: one scale block

__device__ __forceinline__ void to_lds(const uint8_t* g, uint8_t* l) {
    __builtin_amdgcn_global_load_lds(
        (const __attribute__((address_space(1))) void*)g,
        (__attribute__((address_space(3))) void*)l, 16, 0, 0);
}

// Rows of `R` (a multiple of 8 * WAVES) by 128 bytes into LDS.  A wave's
// instruction fills 8 rows; LDS takes lanes in order, so lane l lands on row
// l / 8, 16-byte slot l % 8.  Slot s of row r holds bytes 16 (s ^ (r % 8)),
// which spreads the fragments' reads (16 rows, one slot) over the banks.
template <int R, int WAVES>
struct Stage {
    static constexpr int kLoads = R / 8 / WAVES;
    uint32_t off[kLoads];
    __device__ __forceinline__ void init(int64_t ld, int last_row) {
        const int wave = threadIdx.x / 64, l = threadIdx.x % 64;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            int r = (i * WAVES + wave) * 8 + l / 8;
            const int slot = (l % 8) ^ (r % 8);
            r = r < last_row ? r : last_row;  // rows behind the matrix repeat its last
            off[i] = static_cast<uint32_t>(r) * static_cast<uint32_t>(ld) + 16u * slot;
        }
    }
    __device__ __forceinline__ void load(const uint8_t* base, uint8_t* lds) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            to_lds(base + off[i], lds + (i * WAVES + wave) * 8 * kStep);
    }
};

__device__ __forceinline__ v8i fragment(const uint8_t* lds, int row, int group) {
    const uint8_t* at = lds + row * kStep;
    const int x = row % 8;
    const u32x4 lo = *reinterpret_cast<const u32x4*>(at + 16 * (group ^ x));
    const u32x4 hi = *reinterpret_cast<const u32x4*>(at + 16 * ((group + 4) ^ x));
    v8i r;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        r[k] = static_cast<int>(lo[k]);
        r[k + 4] = static_cast<int>(hi[k]);
    }
    return r;
}

template <int BM, int BN, int WM, int WN, int FA, int FB>
__global__ __launch_bounds__(64 * WM * WN) void q8_gemm_kernel(const GemmArgs a, int tiles_m,
                                                               int tiles_n) {
    constexpr int kWaves = WM * WN;
    constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
    __shared__ __attribute__((aligned(16))) uint8_t lds_a[2][BM * kStep];
    __shared__ __attribute__((aligned(16))) uint8_t lds_b[2][BN * kStep];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l = threadIdx.x % 64;
    const int wm = wave / WN, wn = wave % WN;
    const int64_t m0 = static_cast<int64_t>(blockIdx.x % tiles_m) * BM;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x / tiles_m) * BN;
    const int last_m = static_cast<int>(a.m - 1 - m0 < BM ? a.m - 1 - m0 : BM);
    const int last_n = static_cast<int>(a.n - 1 - n0 < BN ? a.n - 1 - n0 : BN);
    const uint8_t* base_a = a.a + m0 * a.ld_a;
    const uint8_t* base_b = a.b + n0 * a.ld_b;
    Stage<BM, kWaves> stage_a;
    Stage<BN, kWaves> stage_b;
    stage_a.init(a.ld_a, last_m);
    stage_b.init(a.ld_b, last_n);

    // each lane's rows of the scales
    const uint8_t* sa[MI];
    const uint8_t* sb[NI];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        int r = wm * (BM / WM) + 16 * i + l % 16;
        r = r < last_m ? r : last_m;
        sa[i] = a.sa + (m0 + r) * a.ld_sa;
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) {
        int r = wn * (BN / WN) + 16 * j + l % 16;
        r = r < last_n ? r : last_n;
        sb[j] = a.sb + (n0 + r) * a.ld_sb;
    }
    v4f acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = v4f{0, 0, 0, 0};

    const int steps = a.kblocks;
    if (steps > 0) {
        stage_a.load(base_a, lds_a[0]);
        stage_b.load(base_b, lds_b[0]);
    }
    for (int k = 0; k < steps; ++k) {
        __syncthreads();  // step k has landed, and nobody reads the other buffers any more
        const int cur = k & 1;
        if (k + 1 < steps) {
            stage_a.load(base_a + static_cast<int64_t>(k + 1) * kStep, lds_a[cur ^ 1]);
            stage_b.load(base_b + static_cast<int64_t>(k + 1) * kStep, lds_b[cur ^ 1]);
        }
        v8i fb[NI];
        int eb[NI];
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            fb[j] = fragment(lds_b[cur], wn * (BN / WN) + 16 * j + l % 16, l / 16);
            eb[j] = sb[j][k];
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const v8i fa = fragment(lds_a[cur], wm * (BM / WM) + 16 * i + l % 16, l / 16);
            const int ea = sa[i][k];
#pragma unroll
            for (int j = 0; j < NI; ++j)
                // b's rows first: a lane then holds four neighbouring columns of c
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    fb[j], fa, acc[i][j], FB, FA, 0, eb[j], 0, ea);
        }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int64_t row = m0 + wm * (BM / WM) + 16 * i + l % 16;
        if (row >= a.m) continue;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int64_t col = n0 + wn * (BN / WN) + 16 * j + 4 * (l / 16);
            const int64_t at = row * a.ld_c + col;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (col + r < a.n) {
                    float v = acc[i][j][r];
                    if (a.accumulate) v += load1(a.c, at + r, a.c_dtype);
                    store1(a.c, at + r, a.c_dtype, v);
                }
        }
    }
}

template <int BM, int BN, int WM, int WN>
hipError_t gemm_formats(const GemmArgs& a, hipStream_t stream) {
    const int tm = static_cast<int>((a.m + BM - 1) / BM), tn = static_cast<int>((a.n + BN - 1) / BN);
    const dim3 grid(static_cast<uint32_t>(static_cast<int64_t>(tm) * tn)), block(64 * WM * WN);
    if (a.fmt_a == ZERO_E4M3) {
        if (a.fmt_b == ZERO_E4M3)
            q8_gemm_kernel<BM, BN, WM, WN, 0, 0><<<grid, block, 0, stream>>>(a, tm, tn);
        else q8_gemm_kernel<BM, BN, WM, WN, 0, 1><<<grid, block, 0, stream>>>(a, tm, tn);
    } else {
        if (a.fmt_b == ZERO_E4M3)
            q8_gemm_kernel<BM, BN, WM, WN, 1, 0><<<grid, block, 0, stream>>>(a, tm, tn);
        else q8_gemm_kernel<BM, BN, WM, WN, 1, 1><<<grid, block, 0, stream>>>(a, tm, tn);
    }
    return hipGetLastError();
}

}  // namespace

int64_t gemm_blocks(int64_t m, int64_t n, int32_t kblocks) {
    (void)kblocks;
    return (m + 127) / 128 * ((n + 127) / 128);
}

hipError_t launch_q8_gemm(const GemmArgs& a, hipStream_t stream) {
    return gemm_formats<128, 128, 2, 2>(a, stream);
}

}  // namespace zero
