// C ABI of the 8-bit matrices: argument checks, then the launches.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <string>

#include "../../include/fsdp_shard.h"
#include "q8.hpp"
#include "state.hpp"

namespace {

using fsdp::kQ8Block;
using fsdp::kQ8MaxSide;
using fsdp::Q8Mat;
using fsdp::set_error;

bool misaligned(const void *p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0;
}

// A stretch of memory: all of its bytes, or rows of `width` of them, `pitch` apart.
struct Span {
    const void *p;
    int64_t bytes;
    const char *name;
    int64_t width = 0, pitch = 0;
};

bool overlap(const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    if (a.bytes <= 0 || b.bytes <= 0 || x >= y + static_cast<uintptr_t>(b.bytes) ||
        y >= x + static_cast<uintptr_t>(a.bytes))
        return false;
    if (a.pitch == 0 || a.pitch != b.pitch) return true;
    // side by side in the same rows: b starts after a's part of a row and ends with it
    const uintptr_t pitch = static_cast<uintptr_t>(a.pitch);
    const uintptr_t from = y >= x ? (y - x) % pitch : (pitch - (x - y) % pitch) % pitch;
    return from < static_cast<uintptr_t>(a.width) || from + static_cast<uintptr_t>(b.width) > pitch;
}

int64_t down(int64_t n) { return (n + kQ8Block - 1) / kQ8Block; }

// rows of `cols` elements, each `ld` after the other
int64_t extent(int64_t rows, int64_t cols, int64_t ld, int64_t elem) {
    return rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * elem : 0;
}

struct Lines {
    int64_t n, length;
};
Lines scale_lines(const fsdp_q8_t &q) {
    if (q.rows == 0 || q.cols == 0) return {0, 0};
    switch (q.blocks) {
        case FSDP_Q8_ROWS: return {down(q.cols), q.rows};
        case FSDP_Q8_COLS: return {down(q.rows), q.cols};
        case FSDP_Q8_TILES: return {down(q.rows), down(q.cols)};
        default: return {0, 0};
    }
}

Span codes_of(const fsdp_q8_t &q, const char *name) {
    return {q.codes, extent(q.rows, q.cols, q.ld, 1), name, q.cols, q.ld};
}
Span scales_of(const fsdp_q8_t &q, const char *name) {
    const Lines l = scale_lines(q);
    return {q.scales, extent(l.n, l.length, q.pitch, 1), name, l.length, q.pitch};
}

fsdp_status bad(fsdp_status s, const char *call, const char *name, const char *what) {
    return set_error(s, std::string(call) + ": " + name + ": " + what);
}

// A matrix by the rules of fsdp_q8_t, and as the kernels take it.
fsdp_status check(const fsdp_q8_t *q, const char *call, const char *name, Q8Mat *out) {
    if (q == nullptr) return bad(FSDP_E_INVAL, call, name, "null");
    if (q->rows < 0 || q->cols < 0) return bad(FSDP_E_INVAL, call, name, "negative size");
    if (q->rows > kQ8MaxSide || q->cols > kQ8MaxSide || q->ld > kQ8MaxSide)
        return bad(FSDP_E_UNSUPPORTED, call, name, "rows, cols or ld above 2^22");
    if (q->ld < q->cols) return bad(FSDP_E_INVAL, call, name, "ld below cols");
    if (q->format != FSDP_Q8_E4M3 && q->format != FSDP_Q8_E5M2)
        return bad(FSDP_E_UNSUPPORTED, call, name, "format must be FSDP_Q8_E4M3 or FSDP_Q8_E5M2");
    if (q->blocks < FSDP_Q8_TENSOR || q->blocks > FSDP_Q8_TILES)
        return bad(FSDP_E_UNSUPPORTED, call, name, "unknown blocks");
    if (misaligned(q->divisor, 4)) return bad(FSDP_E_ALIGN, call, name, "divisor not 4-byte aligned");
    const Lines l = scale_lines(*q);
    if (q->blocks != FSDP_Q8_TENSOR && l.n > 0) {
        if (q->pitch < l.length || q->pitch > kQ8MaxSide)
            return bad(FSDP_E_INVAL, call, name, "pitch shorter than a line of scales or above 2^22");
        if (q->scales == nullptr) return bad(FSDP_E_INVAL, call, name, "null scales");
        if (q->blocks != FSDP_Q8_TILES && (misaligned(q->scales, 4) || (q->pitch & 3) != 0))
            return bad(FSDP_E_ALIGN, call, name, "scales or pitch not a multiple of 4 bytes");
    }
    if (q->rows > 0 && q->cols > 0 && q->codes == nullptr)
        return bad(FSDP_E_INVAL, call, name, "null codes");
    *out = {q->codes,
            q->scales,
            q->divisor,
            q->ld,
            q->pitch,
            static_cast<int32_t>(q->rows),
            static_cast<int32_t>(q->cols),
            q->format,
            q->blocks};
    return FSDP_OK;
}

// A bf16 or fp32 matrix.
fsdp_status check_wide(const void *p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                       const char *call, const char *name, Span *span) {
    if (dtype != FSDP_DTYPE_BF16 && dtype != FSDP_DTYPE_F32)
        return bad(FSDP_E_UNSUPPORTED, call, name, "dtype must be FSDP_DTYPE_BF16 or FSDP_DTYPE_F32");
    const int64_t elem = dtype == FSDP_DTYPE_F32 ? 4 : 2;
    if (ld < cols) return bad(FSDP_E_INVAL, call, name, "leading dimension below the row's length");
    if (ld > kQ8MaxSide) return bad(FSDP_E_UNSUPPORTED, call, name, "leading dimension above 2^22");
    *span = {p, extent(rows, cols, ld, elem), name, cols * elem, ld * elem};
    if (span->bytes > 0 && p == nullptr) return bad(FSDP_E_INVAL, call, name, "null");
    if (misaligned(p, static_cast<uintptr_t>(elem)))
        return bad(FSDP_E_ALIGN, call, name, "not aligned to its element");
    return FSDP_OK;
}

// No span of `outs` shares a byte with another of them or with one of `ins`.
template <size_t NO, size_t NI>
fsdp_status check_apart(const Span (&outs)[NO], const Span (&ins)[NI], const char *call) {
    for (size_t i = 0; i < NO; ++i) {
        for (size_t k = i + 1; k < NO; ++k)
            if (overlap(outs[i], outs[k]))
                return bad(FSDP_E_INVAL, call, outs[i].name,
                           (std::string("overlaps ") + outs[k].name).c_str());
        for (size_t k = 0; k < NI; ++k)
            if (overlap(outs[i], ins[k]))
                return bad(FSDP_E_INVAL, call, outs[i].name,
                           (std::string("overlaps ") + ins[k].name).c_str());
    }
    return FSDP_OK;
}

fsdp_status launched(hipError_t e, const char *call) {
    return e == hipSuccess ? FSDP_OK
                           : fsdp::set_hip_error(e, (std::string(call) + ": launch").c_str());
}

// The two matrices of a product and its sizes.
fsdp_status check_product(const fsdp_q8_t *a, int32_t ta, const fsdp_q8_t *b, int32_t tb,
                          const char *call, Q8Mat *A, Q8Mat *B) {
    fsdp_status s = check(a, call, "a", A);
    if (s != FSDP_OK || (s = check(b, call, "b", B)) != FSDP_OK) return s;
    if ((ta != 0 && ta != 1) || (tb != 0 && tb != 1))
        return set_error(FSDP_E_INVAL, std::string(call) + ": trans_a and trans_b are 0 or 1");
    if (ta && tb)
        return set_error(FSDP_E_UNSUPPORTED, std::string(call) + ": both operands transposed");
    if (b->format != FSDP_Q8_E4M3)
        return set_error(FSDP_E_UNSUPPORTED, std::string(call) + ": b must be E4M3");
    // the sum runs along the rows of a (down its columns where it is transposed),
    // and the other way round for b
    const int32_t not_a = ta ? FSDP_Q8_ROWS : FSDP_Q8_COLS;
    const int32_t not_b = tb ? FSDP_Q8_COLS : FSDP_Q8_ROWS;
    if (a->blocks == not_a || b->blocks == not_b)
        return set_error(FSDP_E_UNSUPPORTED,
                         std::string(call) + ": " + (a->blocks == not_a ? "a" : "b") +
                             "'s blocks lie across the sum: along it, or 128 x 128, are needed");
    if ((ta ? a->rows : a->cols) != (tb ? b->cols : b->rows))
        return set_error(FSDP_E_INVAL, std::string(call) + ": the operands' inner sizes differ");
    return FSDP_OK;
}

int64_t bytes_of(const fsdp::Q8Cut &c) { return c.bytes_a + c.bytes_b + c.bytes_sums; }

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// The workspace of a linear layer's two steps: x, or dy both ways round, in 8 bits,
// then what the products need.
struct Linear {
    Q8Mat w{}, x{}, dy{}, dyt{};
    fsdp::Q8Cut forward{}, input{};
    int64_t held = 0, sums = 0;
    char *base = nullptr;
    void *products = nullptr;

    // A quantised [rows, cols] at `at`, which it moves on.
    static Q8Mat matrix(char *&at, int64_t rows, int64_t cols, int32_t format, int32_t blocks) {
        fsdp_q8_t q{};
        q.rows = rows, q.cols = cols, q.ld = up(cols, 16), q.blocks = blocks;
        const Lines l = scale_lines(q);
        Q8Mat m{};
        m.rows = static_cast<int32_t>(rows), m.cols = static_cast<int32_t>(cols);
        m.format = format, m.blocks = blocks;
        m.ld = q.ld, m.pitch = up(l.length, 16);
        m.codes = reinterpret_cast<uint8_t *>(at);
        at += up(rows * m.ld, 256);
        m.scales = reinterpret_cast<uint8_t *>(at);
        at += up(l.n * m.pitch, 256);
        return m;
    }

    // Where everything lies from `from`; the products' memory is the largest that one of
    // the three needs, whatever the alignment of what they are given.
    void lay(char *from, int32_t format) {
        char *at = from;
        x = matrix(at, x.rows, w.cols, FSDP_Q8_E4M3, FSDP_Q8_ROWS);
        const int64_t one = at - from;
        at = from;
        dy = matrix(at, x.rows, w.rows, format, FSDP_Q8_ROWS);
        dyt = matrix(at, x.rows, w.rows, format, FSDP_Q8_COLS);
        held = at - from > one ? at - from : one;
        base = from;
        products = from + held;
    }

    fsdp_status plan(const fsdp_q8_t *W, int64_t tokens, int32_t format, const char *call) {
        fsdp_status s = check(W, call, "w", &w);
        if (s != FSDP_OK) return s;
        if (W->format != FSDP_Q8_E4M3 ||
            (W->blocks != FSDP_Q8_TILES && W->blocks != FSDP_Q8_TENSOR))
            return bad(FSDP_E_UNSUPPORTED, call, "w", "must be E4M3, in TILES or TENSOR");
        if (format != FSDP_Q8_E4M3 && format != FSDP_Q8_E5M2)
            return bad(FSDP_E_UNSUPPORTED, call, "format", "must be FSDP_Q8_E4M3 or FSDP_Q8_E5M2");
        if (tokens < 0) return bad(FSDP_E_INVAL, call, "tokens", "negative");
        if (tokens > kQ8MaxSide || up(w.rows, 16) > kQ8MaxSide || up(w.cols, 16) > kQ8MaxSide)
            return bad(FSDP_E_UNSUPPORTED, call, "tokens", "above 2^22");
        x.rows = static_cast<int32_t>(tokens);
        lay(nullptr, format);
        forward = fsdp::q8_cut(x, false, w, true);
        input = fsdp::q8_cut(dy, false, w, false);
        // a checkpoint at the worst alignment
        Q8Mat odd = x;
        odd.codes = reinterpret_cast<uint8_t *>(uintptr_t{1});
        const int64_t a = bytes_of(forward), b = bytes_of(input),
                      c = bytes_of(fsdp::q8_cut(dyt, true, odd, false));
        sums = a > b ? a : b;
        sums = sums > c ? sums : c;
        fmt = format;
        return FSDP_OK;
    }
    int32_t fmt = 0;

    int64_t bytes() const { return held + sums; }
    Span span() const { return {base, bytes(), "workspace"}; }

    fsdp_status place(void *workspace, int64_t have, const char *call) {
        if (bytes() > 0) {
            if (workspace == nullptr || have < bytes())
                return set_error(FSDP_E_INVAL, std::string(call) + ": the workspace needs " +
                                                   std::to_string(bytes()) + " bytes");
            if (misaligned(workspace, 256))
                return set_error(FSDP_E_ALIGN,
                                 std::string(call) + ": workspace not 256-byte aligned");
        }
        lay(static_cast<char *>(workspace), fmt);
        return FSDP_OK;
    }

    fsdp_status check_saved(const fsdp_q8_t *saved, const char *call, Q8Mat *S) const {
        const fsdp_status s = check(saved, call, "saved", S);
        if (s != FSDP_OK) return s;
        if (saved->format != FSDP_Q8_E4M3 || saved->blocks != FSDP_Q8_COLS)
            return bad(FSDP_E_UNSUPPORTED, call, "saved", "must be E4M3, in COLS");
        if (saved->rows != x.rows || saved->cols != w.cols)
            return bad(FSDP_E_INVAL, call, "saved", "must be [tokens, in]");
        if (saved->divisor != nullptr)
            return bad(FSDP_E_INVAL, call, "saved", "a divisor is for reading only");
        return FSDP_OK;
    }
};

}  // namespace

extern "C" {

fsdp_status fsdp_q8_quantize(const void *x, int32_t dtype, int64_t ldx, const fsdp_q8_t *a,
                             const fsdp_q8_t *b, void *stream) try {
    const char *call = "fsdp_q8_quantize";
    Q8Mat A{}, B{};
    fsdp_status s = check(a, call, "a", &A);
    if (s != FSDP_OK || (b != nullptr && (s = check(b, call, "b", &B)) != FSDP_OK)) return s;
    if (a->blocks == FSDP_Q8_TENSOR)
        return set_error(FSDP_E_UNSUPPORTED, std::string(call) + ": a has no blocks");
    if (a->divisor != nullptr || (b != nullptr && b->divisor != nullptr))
        return set_error(FSDP_E_INVAL, std::string(call) + ": a divisor is for reading only");
    Span X;
    if ((s = check_wide(x, dtype, a->rows, a->cols, ldx, call, "x", &X)) != FSDP_OK) return s;
    if (b != nullptr) {
        if (a->rows != b->rows || a->cols != b->cols || a->format != b->format)
            return set_error(FSDP_E_INVAL, std::string(call) + ": a and b differ in size or format");
        if (!((a->blocks == FSDP_Q8_ROWS && b->blocks == FSDP_Q8_COLS) ||
              (a->blocks == FSDP_Q8_COLS && b->blocks == FSDP_Q8_ROWS)))
            return set_error(FSDP_E_UNSUPPORTED,
                             std::string(call) + ": two outputs are one of ROWS and one of COLS");
        const Span outs[4] = {codes_of(*a, "a's codes"), scales_of(*a, "a's scales"),
                              codes_of(*b, "b's codes"), scales_of(*b, "b's scales")};
        const Span ins[1] = {X};
        s = check_apart(outs, ins, call);
    } else {
        const Span outs[2] = {codes_of(*a, "a's codes"), scales_of(*a, "a's scales")};
        const Span ins[1] = {X};
        s = check_apart(outs, ins, call);
    }
    if (s != FSDP_OK) return s;
    hipError_t e = fsdp::injected_fault();
    if (e == hipSuccess)
        e = fsdp::launch_q8_quantize(x, dtype == FSDP_DTYPE_F32, ldx, A, b ? &B : nullptr,
                                     static_cast<hipStream_t>(stream));
    return launched(e, call);
} catch (...) {
    return FSDP_E_NOMEM;
}

fsdp_status fsdp_q8_dequantize(const fsdp_q8_t *q, void *out, int32_t dtype, int64_t ldo,
                               void *stream) try {
    const char *call = "fsdp_q8_dequantize";
    Q8Mat Q{};
    Span O;
    fsdp_status s = check(q, call, "q", &Q);
    if (s != FSDP_OK ||
        (s = check_wide(out, dtype, q->rows, q->cols, ldo, call, "out", &O)) != FSDP_OK)
        return s;
    const Span outs[1] = {O};
    const Span ins[3] = {codes_of(*q, "q's codes"), scales_of(*q, "q's scales"),
                         {q->divisor, q->divisor ? 4 : 0, "q's divisor"}};
    if ((s = check_apart(outs, ins, call)) != FSDP_OK) return s;
    hipError_t e = fsdp::injected_fault();
    if (e == hipSuccess)
        e = fsdp::launch_q8_dequantize(Q, out, dtype == FSDP_DTYPE_F32, ldo,
                                       static_cast<hipStream_t>(stream));
    return launched(e, call);
} catch (...) {
    return FSDP_E_NOMEM;
}

fsdp_status fsdp_q8_product_workspace(const fsdp_q8_t *a, int32_t trans_a, const fsdp_q8_t *b,
                                      int32_t trans_b, int64_t *bytes) try {
    const char *call = "fsdp_q8_product_workspace";
    Q8Mat A{}, B{};
    fsdp_status s = check_product(a, trans_a, b, trans_b, call, &A, &B);
    if (s != FSDP_OK) return s;
    if (bytes == nullptr) return set_error(FSDP_E_INVAL, std::string(call) + ": null bytes");
    *bytes = bytes_of(fsdp::q8_cut(A, trans_a != 0, B, trans_b != 0));
    return FSDP_OK;
} catch (...) {
    return FSDP_E_NOMEM;
}

fsdp_status fsdp_q8_product_cut(const fsdp_q8_t *a, int32_t trans_a, const fsdp_q8_t *b,
                                int32_t trans_b, int32_t *tile, int32_t *split) try {
    const char *call = "fsdp_q8_product_cut";
    Q8Mat A{}, B{};
    fsdp_status s = check_product(a, trans_a, b, trans_b, call, &A, &B);
    if (s != FSDP_OK) return s;
    if (tile == nullptr || split == nullptr)
        return set_error(FSDP_E_INVAL, std::string(call) + ": null tile or split");
    const fsdp::Q8Cut cut = fsdp::q8_cut(A, trans_a != 0, B, trans_b != 0);
    *tile = fsdp::kQ8TileSide[cut.tile];
    *split = cut.split;
    return FSDP_OK;
} catch (...) {
    return FSDP_E_NOMEM;
}

fsdp_status fsdp_q8_product(const fsdp_q8_t *a, int32_t trans_a, const fsdp_q8_t *b,
                            int32_t trans_b, uint16_t *out, int64_t ldo, void *workspace,
                            int64_t workspace_bytes, void *stream) try {
    const char *call = "fsdp_q8_product";
    Q8Mat A{}, B{};
    fsdp_status s = check_product(a, trans_a, b, trans_b, call, &A, &B);
    if (s != FSDP_OK) return s;
    const int64_t M = trans_a ? a->cols : a->rows, N = trans_b ? b->rows : b->cols;
    Span O;
    if ((s = check_wide(out, FSDP_DTYPE_BF16, M, N, ldo, call, "out", &O)) != FSDP_OK) return s;
    const fsdp::Q8Cut cut = fsdp::q8_cut(A, trans_a != 0, B, trans_b != 0);
    const int64_t need = bytes_of(cut);
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < need)
            return set_error(FSDP_E_INVAL, std::string(call) + ": the workspace needs " +
                                               std::to_string(need) + " bytes");
        if (misaligned(workspace, 256))
            return set_error(FSDP_E_ALIGN, std::string(call) + ": workspace not 256-byte aligned");
    }
    const Span outs[2] = {O, {workspace, need, "workspace"}};
    const Span ins[6] = {codes_of(*a, "a's codes"),
                         scales_of(*a, "a's scales"),
                         codes_of(*b, "b's codes"),
                         scales_of(*b, "b's scales"),
                         {a->divisor, a->divisor ? 4 : 0, "a's divisor"},
                         {b->divisor, b->divisor ? 4 : 0, "b's divisor"}};
    if ((s = check_apart(outs, ins, call)) != FSDP_OK) return s;
    hipError_t e = fsdp::injected_fault();
    if (e == hipSuccess)
        e = fsdp::launch_q8_product(A, trans_a != 0, B, trans_b != 0, out, ldo, cut, workspace,
                                    static_cast<hipStream_t>(stream));
    return launched(e, call);
} catch (...) {
    return FSDP_E_NOMEM;
}

fsdp_status fsdp_q8_linear_workspace(const fsdp_q8_t *w, int64_t tokens, int64_t *bytes) try {
    const char *call = "fsdp_q8_linear_workspace";
    if (bytes == nullptr) return set_error(FSDP_E_INVAL, std::string(call) + ": null bytes");
    Linear l;
    const fsdp_status s = l.plan(w, tokens, FSDP_Q8_E4M3, call);
    if (s == FSDP_OK) *bytes = l.bytes();
    return s;
} catch (...) {
    return FSDP_E_NOMEM;
}

fsdp_status fsdp_q8_linear_forward(const fsdp_q8_t *w, const void *x, int32_t dtype, int64_t ldx,
                                   int64_t tokens, const fsdp_q8_t *saved, uint16_t *y, int64_t ldy,
                                   void *workspace, int64_t workspace_bytes, void *stream) try {
    const char *call = "fsdp_q8_linear_forward";
    Linear l;
    Q8Mat S{};
    Span X, Y;
    fsdp_status s = l.plan(w, tokens, FSDP_Q8_E4M3, call);
    if (s != FSDP_OK || (saved != nullptr && (s = l.check_saved(saved, call, &S)) != FSDP_OK) ||
        (s = check_wide(x, dtype, tokens, w->cols, ldx, call, "x", &X)) != FSDP_OK ||
        (s = check_wide(y, FSDP_DTYPE_BF16, tokens, w->rows, ldy, call, "y", &Y)) != FSDP_OK ||
        (s = l.place(workspace, workspace_bytes, call)) != FSDP_OK)
        return s;
    const Span outs[4] = {Y, l.span(), saved ? codes_of(*saved, "saved's codes") : Span{},
                          saved ? scales_of(*saved, "saved's scales") : Span{}};
    const Span ins[4] = {X, codes_of(*w, "w's codes"), scales_of(*w, "w's scales"),
                         {w->divisor, w->divisor ? 4 : 0, "w's divisor"}};
    if ((s = check_apart(outs, ins, call)) != FSDP_OK) return s;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = fsdp::injected_fault();
    if (e == hipSuccess)
        e = fsdp::launch_q8_quantize(x, dtype == FSDP_DTYPE_F32, ldx, l.x, saved ? &S : nullptr, st);
    if (e == hipSuccess) e = fsdp::injected_fault();
    if (e == hipSuccess)
        e = fsdp::launch_q8_product(l.x, false, l.w, true, y, ldy, l.forward, l.products, st);
    return launched(e, call);
} catch (...) {
    return FSDP_E_NOMEM;
}

fsdp_status fsdp_q8_linear_backward(const fsdp_q8_t *w, const fsdp_q8_t *saved, const void *dy,
                                    int32_t dtype, int64_t lddy, int32_t format, uint16_t *dx,
                                    int64_t lddx, uint16_t *dw, int64_t lddw, void *workspace,
                                    int64_t workspace_bytes, void *stream) try {
    const char *call = "fsdp_q8_linear_backward";
    if (saved == nullptr) return bad(FSDP_E_INVAL, call, "saved", "null");
    Linear l;
    Q8Mat S{};
    Span DY, DX{}, DW{};
    const int64_t tokens = saved->rows;
    fsdp_status s = l.plan(w, tokens, format, call);
    if (s != FSDP_OK || (s = l.check_saved(saved, call, &S)) != FSDP_OK ||
        (s = check_wide(dy, dtype, tokens, w->rows, lddy, call, "dy", &DY)) != FSDP_OK ||
        (dx != nullptr && (s = check_wide(dx, FSDP_DTYPE_BF16, tokens, w->cols, lddx, call, "dx",
                                          &DX)) != FSDP_OK) ||
        (dw != nullptr && (s = check_wide(dw, FSDP_DTYPE_BF16, w->rows, w->cols, lddw, call, "dW",
                                          &DW)) != FSDP_OK) ||
        (s = l.place(workspace, workspace_bytes, call)) != FSDP_OK)
        return s;
    const Span outs[3] = {DX, DW, l.span()};
    const Span ins[6] = {DY,
                         codes_of(*w, "w's codes"),
                         scales_of(*w, "w's scales"),
                         {w->divisor, w->divisor ? 4 : 0, "w's divisor"},
                         codes_of(*saved, "saved's codes"),
                         scales_of(*saved, "saved's scales")};
    if ((s = check_apart(outs, ins, call)) != FSDP_OK) return s;
    if (dx == nullptr && dw == nullptr) return FSDP_OK;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const Q8Mat &first = dx ? l.dy : l.dyt;
    hipError_t e = fsdp::injected_fault();
    if (e == hipSuccess)
        e = fsdp::launch_q8_quantize(dy, dtype == FSDP_DTYPE_F32, lddy, first,
                                     dx && dw ? &l.dyt : nullptr, st);
    if (e == hipSuccess && dx != nullptr) {
        e = fsdp::injected_fault();
        if (e == hipSuccess)
            e = fsdp::launch_q8_product(l.dy, false, l.w, false, dx, lddx, l.input, l.products, st);
    }
    if (e == hipSuccess && dw != nullptr) {
        e = fsdp::injected_fault();
        if (e == hipSuccess)
            e = fsdp::launch_q8_product(l.dyt, true, S, false, dw, lddw,
                                        fsdp::q8_cut(l.dyt, true, S, false), l.products, st);
    }
    return launched(e, call);
} catch (...) {
    return FSDP_E_NOMEM;
}

fsdp_status fsdp_plan_block_scales(const fsdp_plan *p, int32_t i, int64_t *offset,
                                   int64_t *total) try {
    const char *call = "fsdp_plan_block_scales";
    if (p == nullptr || offset == nullptr || total == nullptr)
        return set_error(FSDP_E_INVAL, std::string(call) + ": null argument");
    const int32_t n = static_cast<int32_t>(p->L.entries.size());
    // a group of no parameters has no bytes; i counts from 0 all the same
    if (i < 0 || (i >= n && !(n == 0 && i == 0)))
        return set_error(FSDP_E_INVAL, std::string(call) + ": index out of range");
    *offset = *total = 0;
    for (int32_t k = 0; k < n; ++k) {
        if (k == i) *offset = *total;
        *total += down(p->L.entries[k].rows) * down(p->L.entries[k].cols);
    }
    return FSDP_OK;
} catch (...) {
    return FSDP_E_NOMEM;
}

}  // extern "C"

namespace {

// The scales' buffer, and that it is apart from the master shards.
fsdp_status check_scales(const fsdp_plan *p, const uint8_t *scales, const char *call) {
    if (scales == nullptr && p->n_block_scales > 0)
        return set_error(FSDP_E_INVAL, std::string(call) + ": null scales");
    return FSDP_OK;
}

fsdp_status check_shards(const fsdp_plan *p, const Span &buf, const char *call) {
    for (size_t i = 0; i < p->L.entries.size(); ++i) {
        const Span shard{p->host_entries[i].master, p->L.entries[i].valid_numel * 4, "master"};
        if (overlap(buf, shard))
            return set_error(FSDP_E_INVAL, std::string(call) + ": " + buf.name +
                                               " overlaps the master shard of parameter " +
                                               std::to_string(i));
    }
    return FSDP_OK;
}

}  // namespace

extern "C" {

fsdp_status fsdp_block_scales_shard(const fsdp_plan *p, uint8_t *scales, void *stream) try {
    const char *call = "fsdp_block_scales_shard";
    fsdp_status s = fsdp::check_roles(p, FSDP_ROLE_MASTER, call);
    if (s != FSDP_OK || (s = check_scales(p, scales, call)) != FSDP_OK ||
        (s = check_shards(p, {scales, p->n_block_scales, "scales"}, call)) != FSDP_OK ||
        (s = fsdp::check_plan_device(p)) != FSDP_OK)
        return s;
    hipError_t e = fsdp::injected_fault();
    if (e == hipSuccess)
        e = fsdp::launch_block_scales(p->d_cells, p->n_cells, p->d_blocks, p->d_entries, scales,
                                      static_cast<hipStream_t>(stream));
    return launched(e, call);
} catch (...) {
    return FSDP_E_NOMEM;
}

fsdp_status fsdp_pack_allgather_fp8_blocks(const fsdp_plan *p, uint8_t *ag_in,
                                           const uint8_t *scales, void *stream) try {
    const char *call = "fsdp_pack_allgather_fp8_blocks";
    fsdp_status s = fsdp::check_roles(p, FSDP_ROLE_MASTER, call);
    if (s != FSDP_OK) return s;
    if (ag_in == nullptr && p->L.S > 0)
        return set_error(FSDP_E_INVAL, std::string(call) + ": null ag_in");
    const Span seg{ag_in, p->L.S, "ag_in"};
    if ((s = check_scales(p, scales, call)) != FSDP_OK || (s = check_shards(p, seg, call)) != FSDP_OK)
        return s;
    if (overlap(seg, {scales, p->n_block_scales, "scales"}))
        return set_error(FSDP_E_INVAL, std::string(call) + ": ag_in overlaps scales");
    if ((s = fsdp::check_plan_device(p)) != FSDP_OK) return s;
    hipError_t e = fsdp::injected_fault();
    if (e == hipSuccess)
        e = fsdp::launch_pack_fp8_blocks(p->d_pack, static_cast<int64_t>(p->L.pack.size()),
                                         p->d_blocks, p->d_entries, ag_in, scales,
                                         static_cast<hipStream_t>(stream));
    return launched(e, call);
} catch (...) {
    return FSDP_E_NOMEM;
}

}  // extern "C"
