// Host-only harness of zero_model.h's C-ABI layer (zero_model_abi.cpp), built with g++
// under AddressSanitizer and UndefinedBehaviorSanitizer, and under ThreadSanitizer for
// concurrent calls.  The device side is replaced by stubs that check what each launch
// would receive: whatever the host layer accepts, from arguments drawn over their whole
// ranges, must be arrays that exist, are aligned, whose last byte can be addressed, and
// that the call may write without touching what it reads.  Device pointers are fake.
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
#include "zero_model_internal.h"

namespace {

// embed, its backward, layer norm, its backward, act, its backward, logprob, its backward
std::atomic<long> g_launches[8];

[[noreturn]] void die(const char* what, int line) {
    fprintf(stderr, "FAIL line %d: %s\n", line, what);
    exit(1);
}
#define EXPECT(c)                    \
    do {                             \
        if (!(c)) die(#c, __LINE__); \
    } while (0)

// An array of one call, in 128 bits.
struct Span {
    unsigned __int128 lo, hi, row, stride;
};
Span span(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size, uintptr_t align) {
    EXPECT(p != nullptr);
    EXPECT(reinterpret_cast<uintptr_t>(p) % align == 0);
    EXPECT(rows > 0 && cols > 0 && ld >= cols);
    const unsigned __int128 lo = reinterpret_cast<uintptr_t>(p), one = static_cast<uint64_t>(size);
    const unsigned __int128 n =
        (static_cast<unsigned __int128>(rows - 1) * static_cast<uint64_t>(ld) +
         static_cast<uint64_t>(cols)) * one;
    EXPECT(n < (static_cast<unsigned __int128>(1) << 60));
    return {lo, lo + n, static_cast<uint64_t>(cols) * one, static_cast<uint64_t>(ld) * one};
}
int64_t size_of(int dtype) {
    EXPECT(dtype >= 0 && dtype <= 2);
    return dtype == ZERO_F32 ? 4 : 2;
}
Span elements(const void* p, int64_t rows, int64_t cols, int64_t ld, int dtype) {
    const int64_t size = size_of(dtype);
    return span(p, rows, cols, ld, size, static_cast<uintptr_t>(size));
}
Span floats(const void* p, int64_t n) { return span(p, 1, n, n, 4, 4); }

// No byte in common: one behind the other, or different columns of one matrix, row by
// row (of the rows that reach the other's range, at most two bands of columns).
bool apart(const Span& a, const Span& b) {
    if (a.hi <= b.lo || b.hi <= a.lo) return true;
    if (a.stride != b.stride) return false;
    const unsigned __int128 d = (b.lo % a.stride + a.stride - a.lo % a.stride) % a.stride;
    return d >= a.row && d + b.row <= a.stride;
}
void all_apart(const std::vector<Span>& out) {
    for (size_t i = 0; i < out.size(); ++i)
        for (size_t j = i + 1; j < out.size(); ++j) EXPECT(apart(out[i], out[j]));
}
void q8(std::vector<Span>* to, const void* q, int64_t ld, const uint8_t* s, int64_t ld_s,
        int64_t rows, int64_t cols) {
    const int64_t b = (cols + 127) / 128;
    to->push_back(span(q, rows, 128 * b, ld, 1, 16));
    EXPECT(ld % 16 == 0 && ld_s % 4 == 0);
    to->push_back(span(s, rows, (b + 3) / 4 * 4, ld_s, 1, 4));
}
bool same(const void* a, int64_t lda, int ta, const void* b, int64_t ldb, int tb) {
    return a == b && lda == ldb && ta == tb;
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

int64_t embed_blocks(int64_t tokens, int64_t cols) { return tokens * ((cols + 4095) / 4096); }
EmbedWorkspace embed_workspace(int64_t tokens, int64_t cols) {
    EmbedWorkspace w = {};
    w.bytes = 20 * tokens + (tokens + 15) / 16 * 8 * cols;
    return w;
}
int64_t embed_backward_blocks(int64_t tokens, int64_t vocab, int64_t cols, int64_t, int32_t) {
    return (tokens + 15) / 16 + (vocab + 7) / 8 * ((cols + 8191) / 8192);
}
int32_t layernorm_backward_parts(int64_t rows, int32_t) {
    return static_cast<int32_t>(rows < 256 ? rows : 256);
}
int64_t act_blocks(int64_t rows, int64_t cols) { return (rows + 15) / 16 * ((cols + 2047) / 2048); }
int64_t logprob_backward_blocks(int64_t rows, int64_t vocab) {
    return rows * ((vocab + 8191) / 8192);
}

hipError_t launch_embed(const EmbedArgs& a, hipStream_t) {
    ++g_launches[0];
    EXPECT(a.vocab >= 1 && a.vocab <= 0x7fffffff && a.cols >= 1 && a.cols <= 0x7fffffff);
    const Span y = elements(a.y, a.tokens, a.cols, a.ld_y, a.y_dtype);
    EXPECT(apart(y, elements(a.table[0], a.vocab, a.cols, a.ld_t, a.t_dtype)));
    if (a.ctl) EXPECT(apart(y, elements(a.table[1], a.vocab, a.cols, a.ld_t, a.t_dtype)));
    EXPECT(a.id_bytes == 4 || a.id_bytes == 8);
    EXPECT(apart(y, span(a.ids, 1, a.tokens, a.tokens, a.id_bytes,
                         static_cast<uintptr_t>(a.id_bytes))));
    return hipSuccess;
}

hipError_t launch_embed_backward(const EmbedBackwardArgs& a, hipStream_t) {
    ++g_launches[1];
    EXPECT(a.tokens >= 0 && a.tokens <= ZERO_EMBED_MAX_TOKENS);
    std::vector<Span> out = {elements(a.dtable, a.vocab, a.cols, a.ld_dt, a.dt_dtype)};
    if (a.tokens > 0) {
        const int64_t n = embed_workspace(a.tokens, a.cols).bytes;
        out.push_back(span(a.workspace, 1, n, n, 1, 16));
        const Span dy = elements(a.dy, a.tokens, a.cols, a.ld_dy, a.dy_dtype);
        const Span ids = span(a.ids, 1, a.tokens, a.tokens, a.id_bytes,
                              static_cast<uintptr_t>(a.id_bytes));
        for (const Span& o : out) EXPECT(apart(o, dy) && apart(o, ids));
    }
    all_apart(out);
    return hipSuccess;
}

hipError_t launch_layernorm(const LayerNormArgs& a, hipStream_t) {
    ++g_launches[2];
    EXPECT(a.cols >= 1 && a.cols <= ZERO_LAYERNORM_MAX_COLS && a.rows <= 0x7fffffff);
    const Span x = elements(a.x, a.rows, a.cols, a.ld_x, a.x_dtype);
    std::vector<Span> in = {elements(a.weight, 1, a.cols, a.cols, a.w_dtype)}, out;
    if (a.bias) in.push_back(elements(a.bias, 1, a.cols, a.cols, a.w_dtype));
    if (a.h) {
        EXPECT(a.res);
        out.push_back(elements(a.h, a.rows, a.cols, a.ld_h, a.r_dtype));
        EXPECT(apart(out.back(), x) || same(a.h, a.ld_h, a.r_dtype, a.x, a.ld_x, a.x_dtype));
        EXPECT(apart(out.back(), elements(a.res, a.rows, a.cols, a.ld_r, a.r_dtype)) ||
               same(a.h, a.ld_h, a.r_dtype, a.res, a.ld_r, a.r_dtype));
    }
    if (a.y) {
        out.push_back(elements(a.y, a.rows, a.cols, a.ld_y, a.y_dtype));
        EXPECT(apart(out.back(), x) || same(a.y, a.ld_y, a.y_dtype, a.x, a.ld_x, a.x_dtype));
        if (a.res)
            EXPECT(apart(out.back(), elements(a.res, a.rows, a.cols, a.ld_r, a.r_dtype)));
    }
    const size_t matrices = out.size();
    if (a.q) q8(&out, a.q, a.ld_q, a.s, a.ld_s, a.rows, a.cols);
    if (a.mean) out.push_back(floats(a.mean, a.rows));
    if (a.rstd) out.push_back(floats(a.rstd, a.rows));
    EXPECT(!out.empty());
    for (size_t i = matrices; i < out.size(); ++i) EXPECT(apart(out[i], x));
    for (const Span& o : out)
        for (const Span& i : in) EXPECT(apart(o, i));
    all_apart(out);
    return hipSuccess;
}

hipError_t launch_layernorm_backward(const LayerNormBackwardArgs& a, hipStream_t) {
    ++g_launches[3];
    EXPECT(a.cols >= 1 && a.cols <= ZERO_LAYERNORM_MAX_COLS && a.rows <= 0x7fffffff);
    std::vector<Span> out;
    if (a.dw) out.push_back(elements(a.dw, 1, a.cols, a.cols, a.dw_dtype));
    if (a.db) out.push_back(elements(a.db, 1, a.cols, a.cols, a.dw_dtype));
    EXPECT((a.parts != nullptr) <= (a.dw || a.db));
    if (a.rows > 0) {
        if (a.dw || a.db)
            out.push_back(span(a.parts, 2 * layernorm_backward_parts(a.rows, a.cols), a.cols,
                               a.cols, 4, 16));
        out.push_back(elements(a.dx, a.rows, a.cols, a.ld_dx, a.dx_dtype));
        const Span dy = elements(a.dy, a.rows, a.cols, a.ld_dy, a.dy_dtype);
        const Span h = elements(a.h, a.rows, a.cols, a.ld_h, a.h_dtype);
        std::vector<Span> in = {elements(a.weight, 1, a.cols, a.cols, a.w_dtype),
                                floats(a.mean, a.rows), floats(a.rstd, a.rows)};
        EXPECT(apart(out.back(), dy) || same(a.dx, a.ld_dx, a.dx_dtype, a.dy, a.ld_dy, a.dy_dtype));
        EXPECT(apart(out.back(), h) || same(a.dx, a.ld_dx, a.dx_dtype, a.h, a.ld_h, a.h_dtype));
        for (size_t i = 0; i + 1 < out.size(); ++i) EXPECT(apart(out[i], dy) && apart(out[i], h));
        for (const Span& o : out)
            for (const Span& i : in) EXPECT(apart(o, i));
    }
    all_apart(out);
    return hipSuccess;
}

hipError_t launch_act(const ActArgs& a, hipStream_t) {
    ++g_launches[4];
    EXPECT(a.kind >= 0 && a.kind <= 2);
    std::vector<Span> in = {elements(a.gate, a.rows, a.cols, a.ld_g, a.x_dtype)}, out;
    if (a.up) in.push_back(elements(a.up, a.rows, a.cols, a.ld_u, a.x_dtype));
    if (a.q) q8(&out, a.q, a.ld_q, a.s, a.ld_s, a.rows, a.cols);
    if (a.gate_q) q8(&out, a.gate_q, a.ld_gq, a.gate_s, a.ld_gs, a.rows, a.cols);
    if (a.up_q) {
        EXPECT(a.up);
        q8(&out, a.up_q, a.ld_uq, a.up_s, a.ld_us, a.rows, a.cols);
    }
    for (const Span& o : out)
        for (const Span& i : in) EXPECT(apart(o, i));
    if (a.y) {
        out.push_back(elements(a.y, a.rows, a.cols, a.ld_y, a.y_dtype));
        EXPECT(apart(out.back(), in[0]) || same(a.y, a.ld_y, a.y_dtype, a.gate, a.ld_g, a.x_dtype));
        if (a.up)
            EXPECT(apart(out.back(), in[1]) ||
                   same(a.y, a.ld_y, a.y_dtype, a.up, a.ld_u, a.x_dtype));
    }
    EXPECT(!out.empty());
    all_apart(out);
    return hipSuccess;
}

hipError_t launch_act_backward(const ActBackwardArgs& a, hipStream_t) {
    ++g_launches[5];
    EXPECT(a.kind >= 0 && a.kind <= 2 && !a.up_q == !a.dup);
    const Span dy = elements(a.dy, a.rows, a.cols, a.ld_dy, a.dy_dtype);
    std::vector<Span> in, out;
    q8(&in, a.gate_q, a.ld_gq, a.gate_s, a.ld_gs, a.rows, a.cols);
    if (a.up_q) q8(&in, a.up_q, a.ld_uq, a.up_s, a.ld_us, a.rows, a.cols);
    auto put = [&](const void* p, int64_t ld, int dtype) {
        out.push_back(elements(p, a.rows, a.cols, ld, dtype));
        EXPECT(apart(out.back(), dy) || same(p, ld, dtype, a.dy, a.ld_dy, a.dy_dtype));
    };
    put(a.dgate, a.ld_dg, a.dx_dtype);
    if (a.dup) put(a.dup, a.ld_du, a.dx_dtype);
    if (a.y) put(a.y, a.ld_y, a.y_dtype);
    for (const Span& o : out)
        for (const Span& i : in) EXPECT(apart(o, i));
    all_apart(out);
    return hipSuccess;
}

hipError_t launch_logprob(const LogprobArgs& a, hipStream_t) {
    ++g_launches[6];
    EXPECT(a.rows >= 1 && a.rows <= 0x7fffffff && a.vocab >= 1 && a.vocab <= 0x7fffffff);
    std::vector<Span> in = {elements(a.logits, a.rows, a.vocab, a.ld, a.dtype)}, out;
    if (a.ids)
        in.push_back(span(a.ids, 1, a.rows, a.rows, a.id_bytes,
                          static_cast<uintptr_t>(a.id_bytes)));
    if (a.logp) {
        EXPECT(a.ids);
        out.push_back(floats(a.logp, a.rows));
    }
    if (a.entropy) out.push_back(floats(a.entropy, a.rows));
    if (a.lse) out.push_back(floats(a.lse, a.rows));
    EXPECT(!a.top_index == !a.top_logit && !a.top_index == (a.top == 0));
    if (a.top_index) {
        EXPECT(a.top >= 1 && a.top <= ZERO_LOGPROB_MAX_TOP);
        out.push_back(span(a.top_index, a.rows, a.top, a.ld_top, 4, 4));
        out.push_back(elements(a.top_logit, a.rows, a.top, a.ld_top, a.dtype));
    }
    EXPECT(!out.empty());
    for (const Span& o : out)
        for (const Span& i : in) EXPECT(apart(o, i));
    all_apart(out);
    return hipSuccess;
}

hipError_t launch_logprob_backward(const LogprobBackwardArgs& a, hipStream_t) {
    ++g_launches[7];
    EXPECT(a.rows >= 1 && a.rows <= 0x7fffffff && a.vocab >= 1 && a.vocab <= 0x7fffffff);
    EXPECT(a.dlogp || a.dentropy);
    const Span x = elements(a.logits, a.rows, a.vocab, a.ld, a.dtype);
    const Span g = elements(a.grad, a.rows, a.vocab, a.ld_grad, a.dtype);
    EXPECT(apart(g, x) || (a.grad == a.logits && a.ld_grad == a.ld));
    EXPECT(apart(g, floats(a.lse, a.rows)));
    if (a.dlogp) {
        EXPECT(a.ids);
        EXPECT(apart(g, floats(a.dlogp, a.rows)));
    }
    if (a.ids)
        EXPECT(apart(g, span(a.ids, 1, a.rows, a.rows, a.id_bytes,
                             static_cast<uintptr_t>(a.id_bytes))));
    if (a.dentropy)
        EXPECT(apart(g, floats(a.dentropy, a.rows)) && apart(g, floats(a.entropy, a.rows)));
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
        return pick({-1, INT64_MIN, INT64_MAX, 65536, 65537, 16777216, 16777217, int64_t{1} << 31,
                     int64_t{1} << 40, int64_t{1} << 56});
    }
    int64_t ld(int64_t cols) {
        if (r() % 6) return cols > 0 && cols < (int64_t{1} << 40) ? (cols + 127) / 128 * 128 : 128;
        return pick({cols, cols == INT64_MIN ? cols : cols - 1, 0, -16, 4, 16, 1000, 4096,
                     INT64_MAX, INT64_MIN});
    }
    int32_t dtype() { return r() % 12 ? static_cast<int32_t>(r() % 3) : static_cast<int32_t>(r()); }
    int32_t fmt() { return r() % 12 ? static_cast<int32_t>(r() % 2) : static_cast<int32_t>(r()); }
    int32_t id_bytes() { return static_cast<int32_t>(pick({4, 8, 4, 8, 4, 8, 2})); }
    void* ptr() {
        if (r() % 16 == 0) return nullptr;
        // a few regions 2^44 bytes apart, sometimes misaligned, sometimes close together
        uintptr_t p = (1 + r() % 40) << 44;
        if (r() % 12 == 0) p += r() % 64;
        if (r() % 6 == 0) p += (r() % 64) * 256;
        return reinterpret_cast<void*>(p);
    }
    void* maybe() { return r() % 3 ? ptr() : nullptr; }
    float real() {
        static const float v[] = {1.0f, 0.5f, 1e-5f, 0.0f, -1.0f, 1e30f, 1e-39f, 2.0f};
        return r() % 16 ? v[r() % 8] : (r() % 2 ? __builtin_inff() : __builtin_nanf(""));
    }
};

void calls(uint64_t seed, int n) {
    Draw d(seed);
    auto u8 = [&] { return static_cast<uint8_t*>(d.ptr()); };
    auto f32 = [&] { return static_cast<float*>(d.ptr()); };
    auto ctl = [&] { return static_cast<zero_step_control*>(d.ptr()); };
    for (int k = 0; k < n; ++k) {
        const int64_t rows = d.dim(), cols = d.dim(), tokens = d.dim();
        zero_embed(d.ptr(), d.dtype(), rows, cols, d.ld(cols), d.ptr(), d.id_bytes(), tokens,
                   d.real(), d.ptr(), d.dtype(), d.ld(cols), nullptr);
        const void* two[2] = {d.ptr(), d.ptr()};
        zero_embed_ctl(d.r() % 16 ? two : nullptr, rows, cols, d.ld(cols), d.ptr(), d.id_bytes(),
                       tokens, d.real(), d.ptr(), d.dtype(), d.ld(cols), ctl(), nullptr);
        int64_t bytes = zero_embed_backward_workspace(tokens, rows, cols);
        EXPECT(bytes >= -1);
        zero_embed_backward(d.ptr(), d.dtype(), d.ld(cols), d.ptr(), d.id_bytes(), tokens, rows,
                            cols, d.real(), d.ptr(), d.dtype(), d.ld(cols),
                            static_cast<int32_t>(d.r() % 3), d.ptr(),
                            d.r() % 4 ? bytes : bytes - 1, nullptr);
        const bool q = d.r() % 2, gq = d.r() % 4, uq = d.r() % 2;
        zero_layernorm(d.ptr(), d.dtype(), d.ld(cols), d.maybe(), d.dtype(), d.ld(cols), d.ptr(),
                       d.maybe(), d.dtype(), rows, cols, d.real(), d.maybe(), d.ld(cols),
                       d.maybe(), d.dtype(), d.ld(cols), q ? d.ptr() : nullptr, d.fmt(),
                       d.ld(cols), q ? u8() : nullptr, d.ld(cols), static_cast<float*>(d.maybe()),
                       static_cast<float*>(d.maybe()), nullptr);
        bytes = zero_layernorm_backward_workspace(rows, cols);
        EXPECT(bytes >= -1 && bytes <= int64_t{8} * 1024 * ZERO_LAYERNORM_MAX_COLS);
        zero_layernorm_backward(d.ptr(), d.dtype(), d.ld(cols), d.ptr(), d.dtype(), d.ld(cols),
                                d.ptr(), d.dtype(), f32(), f32(), d.maybe(), d.dtype(),
                                d.ld(cols), rows, cols, d.ptr(), d.dtype(), d.ld(cols), d.maybe(),
                                d.maybe(), d.dtype(), d.ptr(), d.r() % 4 ? bytes : bytes - 1,
                                nullptr);
        const int32_t kind = d.r() % 12 ? static_cast<int32_t>(d.r() % 3) : 3;
        zero_act(d.ptr(), d.ld(cols), d.maybe(), d.ld(cols), d.dtype(), kind, rows, cols,
                 d.maybe(), d.dtype(), d.ld(cols), q ? d.ptr() : nullptr, d.fmt(), d.ld(cols),
                 q ? u8() : nullptr, d.ld(cols), gq ? d.ptr() : nullptr, d.fmt(), d.ld(cols),
                 gq ? u8() : nullptr, d.ld(cols), uq ? d.ptr() : nullptr, d.ld(cols),
                 uq ? u8() : nullptr, d.ld(cols), nullptr);
        zero_act_backward(d.ptr(), d.dtype(), d.ld(cols), d.ptr(), d.fmt(), d.ld(cols), u8(),
                          d.ld(cols), uq ? d.ptr() : nullptr, d.ld(cols), uq ? u8() : nullptr,
                          d.ld(cols), kind, rows, cols, d.ptr(), d.ld(cols),
                          uq ? d.ptr() : nullptr, d.ld(cols), d.dtype(), d.maybe(), d.dtype(),
                          d.ld(cols), nullptr);
        const int32_t top = static_cast<int32_t>(d.pick({0, 1, 5, 64, 128, 129, -3}));
        zero_logprob(d.ptr(), d.dtype(), d.ld(cols), rows, cols, d.maybe(), d.id_bytes(), d.real(),
                     static_cast<float*>(d.maybe()), static_cast<float*>(d.maybe()),
                     static_cast<float*>(d.maybe()), q ? static_cast<int32_t*>(d.ptr()) : nullptr,
                     q ? d.ptr() : nullptr, top, d.r() % 8 ? top : d.dim(), nullptr);
        zero_logprob_backward(d.ptr(), d.dtype(), d.ld(cols), rows, cols, d.ptr(), d.id_bytes(),
                              d.real(), f32(), static_cast<float*>(d.maybe()), f32(),
                              static_cast<float*>(d.maybe()), d.real(),
                              d.r() % 2 ? ctl() : nullptr, d.ptr(), d.ld(cols), nullptr);
    }
}

}  // namespace

int main(int argc, char** argv) {
    if (argc > 1 && !strcmp(argv[1], "threads")) {
        std::vector<std::thread> t;
        for (int k = 0; k < 8; ++k) t.emplace_back([k] { calls(100 + k, 4000); });
        for (auto& x : t) x.join();
    } else {
        for (uint64_t s = 1; s <= 8; ++s) calls(s, 20000);
    }
    for (auto& n : g_launches) {
        printf("%ld accepted\n", n.load());
        EXPECT(n > 20);
    }
    printf("model harness: ok\n");
    return 0;
}
