// Host-only harness of the training operators' C-ABI layer (zero_train_abi.cpp),
// built with g++ under AddressSanitizer and UndefinedBehaviorSanitizer, and
// under ThreadSanitizer for concurrent calls.  The device side is replaced by
// stubs that check what each launch would receive: whatever the host layer
// accepts, from arguments drawn over their whole ranges, must be arrays that
// exist, are aligned, whose last byte can be addressed, and that the call may
// write without touching what it reads.  Device pointers are fake addresses.
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <atomic>
#include <random>
#include <thread>
#include <vector>

#include "zero_host.h"
#include "zero_train_internal.h"

namespace {

std::atomic<long> g_launches[5];  // quantize, gemm, norm, its backward, distill

[[noreturn]] void die(const char* what, int line) {
    fprintf(stderr, "FAIL line %d: %s\n", line, what);
    exit(1);
}
#define EXPECT(c)                    \
    do {                             \
        if (!(c)) die(#c, __LINE__); \
    } while (0)

struct Span {
    unsigned __int128 lo, hi;
};

// The bytes of rows x cols elements, in 128 bits.
Span span(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size, uintptr_t align) {
    EXPECT(p != nullptr);
    EXPECT(reinterpret_cast<uintptr_t>(p) % align == 0);
    EXPECT(rows > 0 && cols > 0 && ld >= cols);
    const unsigned __int128 lo = reinterpret_cast<uintptr_t>(p);
    const unsigned __int128 n =
        (static_cast<unsigned __int128>(rows - 1) * static_cast<uint64_t>(ld) +
         static_cast<uint64_t>(cols)) * static_cast<uint64_t>(size);
    EXPECT(n < (static_cast<unsigned __int128>(1) << 60));
    return {lo, lo + n};
}
bool apart(const Span& a, const Span& b) { return a.hi <= b.lo || b.hi <= a.lo; }
int64_t size_of(int dtype) {
    EXPECT(dtype >= 0 && dtype <= 2);
    return dtype == ZERO_F32 ? 4 : 2;
}

}  // namespace

namespace zero {

static thread_local char g_error[512];
int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_error, sizeof g_error, fmt, ap);
    va_end(ap);
    return code;
}
int ok() {
    g_error[0] = 0;
    return ZERO_OK;
}
int hip_fail(hipError_t, const char* where) { return fail(ZERO_EHIP, "%s", where); }

int64_t quantize_blocks(int64_t rows, int64_t cols) {
    return (rows + 127) / 128 * ((cols + 127) / 128);
}
int64_t gemm_tiles(int64_t m, int64_t n) { return (m + 63) / 64 * ((n + 63) / 64); }
int32_t norm_backward_parts(int64_t rows, int32_t) {
    return static_cast<int32_t>(rows < 256 ? rows : 256);
}

hipError_t launch_q8_quantize(const QuantizeArgs& a, hipStream_t) {
    ++g_launches[0];
    std::vector<Span> in, out;
    const int64_t bc = (a.cols + 127) / 128, br = (a.rows + 127) / 128;
    in.push_back(span(a.src[0], a.rows, a.cols, a.ld_src, size_of(a.dtype), 2));
    if (a.ctl) in.push_back(span(a.src[1], a.rows, a.cols, a.ld_src, 2, 2));
    EXPECT(a.q || a.qt);
    if (a.q) {
        out.push_back(span(a.q, a.rows, bc * 128, a.ld_q, 1, 16));
        out.push_back(span(a.s, a.rows, (bc + 3) / 4 * 4, a.ld_s, 1, 4));
    }
    if (a.qt) {
        out.push_back(span(a.qt, a.cols, br * 128, a.ld_qt, 1, 16));
        out.push_back(span(a.st, a.cols, (br + 3) / 4 * 4, a.ld_st, 1, 4));
    }
    for (size_t i = 0; i < out.size(); ++i) {
        for (const Span& s : in) EXPECT(apart(out[i], s));
        for (size_t j = i + 1; j < out.size(); ++j) EXPECT(apart(out[i], out[j]));
    }
    return hipSuccess;
}

hipError_t launch_q8_gemm(const GemmArgs& a, hipStream_t) {
    ++g_launches[1];
    const Span c = span(a.c, a.m, a.n, a.ld_c, size_of(a.c_dtype), 2);
    EXPECT(a.kblocks >= 0 && a.kblocks <= ZERO_Q8_MAX_LD / 128);
    // the kernels' 32-bit offsets inside a tile of 256 rows
    EXPECT(255 * a.ld_a + 128 * int64_t{a.kblocks} < (int64_t{1} << 32));
    EXPECT(255 * a.ld_sb + a.kblocks < (int64_t{1} << 32));
    if (a.kblocks) {
        const int64_t k = 128 * int64_t{a.kblocks}, q = (a.kblocks + 3) / 4 * 4;
        EXPECT(apart(c, span(a.a, a.m, k, a.ld_a, 1, 16)));
        EXPECT(apart(c, span(a.b, a.n, k, a.ld_b, 1, 16)));
        EXPECT(apart(c, span(a.sa, a.m, q, a.ld_sa, 1, 4)));
        EXPECT(apart(c, span(a.sb, a.n, q, a.ld_sb, 1, 4)));
    }
    return hipSuccess;
}

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t) {
    ++g_launches[2];
    EXPECT(a.cols >= 1 && a.cols <= ZERO_NORM_MAX_COLS && a.rows <= 0x7fffffff);
    const Span x = span(a.x, a.rows, a.cols, a.ld_x, size_of(a.x_dtype), 2);
    const Span w = span(a.weight, 1, a.cols, a.cols, size_of(a.w_dtype), 2);
    if (a.h) {
        EXPECT(a.res);
        const Span h = span(a.h, a.rows, a.cols, a.ld_h, size_of(a.r_dtype), 2);
        const Span r = span(a.res, a.rows, a.cols, a.ld_r, size_of(a.r_dtype), 2);
        EXPECT(apart(h, w));
        EXPECT(apart(h, x) || (a.h == a.x && a.ld_h == a.ld_x && a.r_dtype == a.x_dtype));
        EXPECT(apart(h, r) || (a.h == a.res && a.ld_h == a.ld_r));
        if (a.y) EXPECT(apart(h, span(a.y, a.rows, a.cols, a.ld_y, size_of(a.y_dtype), 2)));
    }
    if (a.y) {
        const Span y = span(a.y, a.rows, a.cols, a.ld_y, size_of(a.y_dtype), 2);
        EXPECT(apart(y, w));
        EXPECT(apart(y, x) || (a.y == a.x && a.ld_y == a.ld_x && a.y_dtype == a.x_dtype));
        if (a.res)
            EXPECT(apart(y, span(a.res, a.rows, a.cols, a.ld_r, size_of(a.r_dtype), 2)));
    }
    if (a.q) {
        const int64_t b = (a.cols + 127) / 128;
        EXPECT(apart(x, span(a.q, a.rows, 128 * b, a.ld_q, 1, 16)));
        EXPECT(apart(x, span(a.s, a.rows, (b + 3) / 4 * 4, a.ld_s, 1, 4)));
    }
    return hipSuccess;
}

hipError_t launch_rmsnorm_backward(const NormBackwardArgs& a, hipStream_t) {
    ++g_launches[3];
    if (a.rows > 0) {
        const Span dx = span(a.dx, a.rows, a.cols, a.ld_dx, size_of(a.dx_dtype), 2);
        const Span dy = span(a.dy, a.rows, a.cols, a.ld_dy, size_of(a.dy_dtype), 2);
        EXPECT(apart(dx, dy) || (a.dx == a.dy && a.ld_dx == a.ld_dy && a.dx_dtype == a.dy_dtype));
        const Span h = span(a.h, a.rows, a.cols, a.ld_h, size_of(a.h_dtype), 2);
        EXPECT(apart(dx, h) || (a.dx == a.h && a.ld_dx == a.ld_h && a.dx_dtype == a.h_dtype));
        EXPECT(apart(dx, span(a.weight, 1, a.cols, a.cols, size_of(a.w_dtype), 2)));
        EXPECT(apart(dx, span(a.rstd, 1, a.rows, a.rows, 4, 4)));
        if (a.dw) {
            const Span parts = span(a.parts, norm_backward_parts(a.rows, a.cols), a.cols, a.cols,
                                    4, 16);
            EXPECT(apart(parts, dx) && apart(parts, dy) && apart(parts, h));
        }
    }
    return hipSuccess;
}

hipError_t launch_distill(const DistillArgs& a, DistillMode mode, hipStream_t) {
    ++g_launches[4];
    EXPECT(a.rows >= 1 && a.vocab >= 1 && a.vocab <= 0x7fffffff);
    EXPECT(a.top >= 1 && a.top <= ZERO_DISTILL_MAX_TOP);
    const Span x = span(a.logits, a.rows, a.vocab, a.ld, size_of(a.dtype), 2);
    const Span i = span(a.index, a.rows, a.top, a.ld_top, a.index_bytes,
                        static_cast<uintptr_t>(a.index_bytes));
    const Span t = span(a.top_logit, a.rows, a.top, a.ld_top, size_of(a.top_dtype), 2);
    if (mode != kDistillForward) {
        const Span g = span(a.grad, a.rows, a.vocab, a.ld_grad, size_of(a.dtype), 2);
        EXPECT(apart(g, x) || (a.grad == a.logits && a.ld_grad == a.ld));
        EXPECT(apart(g, i) && apart(g, t));
    }
    if (mode == kDistillBackward) span(a.lse_in, 1, a.rows, a.rows, 4, 4);
    return hipSuccess;
}

}  // namespace zero

namespace {

// Values that meet every branch: small and usual ones, borders, extremes.
struct Draw {
    std::mt19937_64 r;
    explicit Draw(uint64_t seed) : r(seed) {}
    int64_t pick(const std::vector<int64_t>& v) { return v[r() % v.size()]; }
    int64_t dim() {
        if (r() % 8) return pick({0, 1, 2, 7, 16, 64, 127, 128, 129, 200, 300, 1000, 4096});
        return pick({-1, INT64_MIN, INT64_MAX, 65536, 65537, int64_t{1} << 31, int64_t{1} << 40,
                     int64_t{1} << 56, 8388608, 8388609});
    }
    int64_t ld(int64_t cols) {
        if (r() % 6) return cols > 0 && cols < (int64_t{1} << 40) ? (cols + 127) / 128 * 128 : 128;
        return pick({cols, cols == INT64_MIN ? cols : cols - 1, 0, -16, 4, 16, 1000, INT64_MAX,
                     INT64_MIN, 8388624});
    }
    int32_t dtype() { return r() % 12 ? static_cast<int32_t>(r() % 3) : static_cast<int32_t>(r()); }
    int32_t fmt() { return r() % 12 ? static_cast<int32_t>(r() % 2) : static_cast<int32_t>(r()); }
    void* ptr() {
        if (r() % 12 == 0) return nullptr;
        // a few regions 2^44 bytes apart, sometimes misaligned, sometimes close together
        uintptr_t p = (1 + r() % 12) << 44;
        if (r() % 8 == 0) p += r() % 64;
        if (r() % 8 == 0) p += (r() % 64) * 1024;
        return reinterpret_cast<void*>(p);
    }
    float real() {
        static const float v[] = {1.0f, 0.5f, 1e-5f, 0.0f, -1.0f, 1e30f, 1e-39f, 2.0f};
        return r() % 16 ? v[r() % 8] : (r() % 2 ? __builtin_inff() : __builtin_nanf(""));
    }
};

void calls(uint64_t seed, int n) {
    Draw d(seed);
    for (int k = 0; k < n; ++k) {
        const int64_t rows = d.dim(), cols = d.dim(), m = d.dim();
        auto u8 = [&] { return static_cast<uint8_t*>(d.ptr()); };
        auto f32 = [&] { return static_cast<float*>(d.ptr()); };
        auto ctl = [&] { return static_cast<zero_step_control*>(d.ptr()); };
        zero_q8_quantize(d.ptr(), d.dtype(), rows, cols, d.ld(cols), d.fmt(), d.ptr(), d.ld(cols),
                         u8(), d.ld(cols), d.ptr(), d.ld(rows), u8(), d.ld(rows), nullptr);
        const void* two[2] = {d.ptr(), d.ptr()};
        zero_q8_quantize_ctl(two, rows, cols, d.ld(cols), d.fmt(), d.ptr(), d.ld(cols), u8(),
                             d.ld(cols), nullptr, 0, nullptr, 0, ctl(), nullptr);
        zero_q8_gemm(d.ptr(), d.fmt(), d.ld(cols), u8(), d.ld(cols), d.ptr(), d.fmt(), d.ld(cols),
                     u8(), d.ld(cols), rows, m, cols, d.ptr(), d.dtype(), d.ld(m),
                     static_cast<int32_t>(d.r() % 3), nullptr);
        zero_rmsnorm(d.ptr(), d.dtype(), d.ld(cols), d.ptr(), d.dtype(), d.ld(cols), d.ptr(),
                     d.dtype(), rows, cols, d.real(), d.ptr(), d.ld(cols), d.ptr(), d.dtype(),
                     d.ld(cols), d.ptr(), d.fmt(), d.ld(cols), u8(), d.ld(cols), f32(), nullptr);
        const int64_t bytes = zero_rmsnorm_backward_workspace(rows, cols);
        EXPECT(bytes >= -1 && bytes <= int64_t{4} * ZERO_NORM_MAX_PARTS * ZERO_NORM_MAX_COLS);
        zero_rmsnorm_backward(d.ptr(), d.dtype(), d.ld(cols), d.ptr(), d.dtype(), d.ld(cols),
                              d.ptr(), d.dtype(), f32(), d.ptr(), d.dtype(), d.ld(cols), rows,
                              cols, d.ptr(), d.dtype(), d.ld(cols), d.ptr(), d.dtype(), d.ptr(),
                              d.r() % 4 ? bytes : bytes - 1, nullptr);
        zero_distill_inputs in;
        memset(&in, 0, sizeof in);
        in.logits = d.ptr(); in.top_index = d.ptr(); in.top_logit = d.ptr(); in.row_weight = f32();
        in.rows = rows; in.vocab = cols; in.ld_logits = d.ld(cols);
        in.top = static_cast<int32_t>(d.pick({0, 1, 5, 64, 128, 1024, 1025, -3}));
        in.ld_top = d.r() % 8 ? in.top : d.dim();
        in.logits_dtype = d.dtype(); in.top_dtype = d.dtype();
        in.index_bytes = static_cast<int32_t>(d.pick({4, 8, 4, 8, 2}));
        in.temperature = d.real();
        const zero_distill_inputs* pin = d.r() % 64 ? &in : nullptr;
        zero_distill_forward(pin, f32(), f32(), nullptr);
        zero_distill_backward(pin, f32(), d.real(), d.r() % 2 ? ctl() : nullptr, d.ptr(),
                              d.ld(cols), nullptr);
        zero_distill(pin, d.real(), d.r() % 2 ? ctl() : nullptr, f32(), f32(), d.ptr(),
                     d.ld(cols), nullptr);
    }
}

}  // namespace

int main(int argc, char** argv) {
    if (argc > 1 && !strcmp(argv[1], "threads")) {
        std::vector<std::thread> t;
        for (int k = 0; k < 8; ++k) t.emplace_back([k] { calls(100 + k, 2000); });
        for (auto& x : t) x.join();
    } else {
        for (uint64_t s = 1; s <= 8; ++s) calls(s, 20000);
    }
    for (auto& n : g_launches) {
        printf("%ld accepted\n", n.load());
        EXPECT(n > 20);
    }
    printf("train harness: ok\n");
    return 0;
}
