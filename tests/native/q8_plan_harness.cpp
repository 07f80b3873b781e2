// What the 8-bit matrices' host code makes and how large, under AddressSanitizer: what a
// bind allocates, and the memory that products need against what their launches touch.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <new>
#include <vector>

#include "../../include/fsdp_shard.h"
#include "q8_harness.hpp"

namespace {
size_t g_allocated = 0;     // bytes asked for since it was last set to 0
size_t g_most = SIZE_MAX;   // an allocation of more fails
}
void *operator new(size_t n) {
    g_allocated += n;
    if (n > g_most) throw std::bad_alloc();
    if (void *p = std::malloc(n > 0 ? n : 1)) return p;
    throw std::bad_alloc();
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, size_t) noexcept { std::free(p); }

namespace {

void must(bool ok, const char *what) {
    if (ok) return;
    std::printf("FAILED %s: %s\n", what, fsdp_last_error());
    std::exit(1);
}

// A bind after the first sends the entries alone: what it allocates follows from the
// parameters' number, not from that of their blocks.
void bind_again() {
    const int64_t rows[2] = {int64_t{1} << 20, 4096}, cols[2] = {1, 4096};
    fsdp_plan *plan = nullptr;
    must(fsdp_plan_create(rows, cols, 2, 1, 0, 1, &plan) == FSDP_OK, "plan");
    std::vector<float *> master;
    for (int i = 0; i < 2; ++i)
        master.push_back(static_cast<float *>(std::malloc(rows[i] * cols[i] * sizeof(float))));
    int64_t at = 0, total = 0;
    must(fsdp_plan_block_scales(plan, 0, &at, &total) == FSDP_OK, "block scales");
    must(total == 8192 + 1024, "blocks");
    std::vector<uint8_t> scales(total);
    // no memory for the blocks: the plan stays as it was
    g_most = static_cast<size_t>(total);
    must(fsdp_bind(plan, master.data(), nullptr, nullptr, nullptr, nullptr, nullptr) == FSDP_E_NOMEM,
         "no memory for the blocks");
    g_most = SIZE_MAX;
    must(fsdp_block_scales_shard(plan, scales.data(), nullptr) == FSDP_E_STATE, "not bound");
    for (int turn = 0; turn < 3; ++turn) {
        g_allocated = 0;
        must(fsdp_bind(plan, master.data(), nullptr, nullptr, nullptr, nullptr, nullptr) == FSDP_OK,
             "bind");
        must(turn == 0 || g_allocated < static_cast<size_t>(total), "a later bind allocates little");
        // and the blocks are those of the first
        for (uint8_t &s : scales) s = 0;
        must(fsdp_block_scales_shard(plan, scales.data(), nullptr) == FSDP_OK, "scales");
        for (uint8_t s : scales) must(s == 2, "every block once");
    }
    fsdp_plan_destroy(plan);
    for (float *p : master) std::free(p);
}

// No exception leaves a C entry, not even where there is no memory for its message.
void out_of_memory() {
    const int64_t rows[1] = {130}, cols[1] = {70};
    fsdp_plan *plan = nullptr;
    must(fsdp_plan_create(rows, cols, 1, 1, 0, 1, &plan) == FSDP_OK, "plan");
    int64_t at = 0, total = 0;
    fsdp_q8_t q{};
    q.rows = -1;
    g_most = 0;
    const fsdp_status got[] = {
        fsdp_plan_block_scales(plan, 7, &at, &total),
        fsdp_plan_block_scales(nullptr, 0, &at, &total),
        fsdp_q8_quantize(&q, FSDP_DTYPE_BF16, 0, &q, nullptr, nullptr),
        fsdp_q8_dequantize(&q, &q, FSDP_DTYPE_BF16, 0, nullptr),
        fsdp_q8_product_workspace(&q, 0, &q, 0, &at),
        fsdp_q8_product(&q, 0, &q, 0, nullptr, 0, nullptr, 0, nullptr),
        fsdp_q8_linear_workspace(&q, 1, &at),
        fsdp_q8_linear_forward(&q, &q, 0, 0, 1, nullptr, nullptr, 0, nullptr, 0, nullptr),
        fsdp_q8_linear_backward(&q, &q, &q, 0, 0, 0, nullptr, 0, nullptr, 0, nullptr, 0, nullptr),
        fsdp_block_scales_shard(plan, nullptr, nullptr),
        fsdp_pack_allgather_fp8_blocks(plan, nullptr, nullptr, nullptr),
    };
    g_most = SIZE_MAX;
    for (fsdp_status s : got) must(s == FSDP_E_NOMEM, "no memory");
    must(fsdp_plan_block_scales(plan, 0, &at, &total) == FSDP_OK && total == 2, "after");
    fsdp_plan_destroy(plan);
}

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t down(int64_t n) { return (n + 127) / 128; }

// A matrix whose codes end with their memory, `at` bytes past a multiple of 256 and rows
// `more` past a multiple of 16 bytes apart.
struct Mat {
    fsdp_q8_t q{};
    std::vector<void *> held;
    Mat(int64_t r, int64_t c, int blocks, int64_t at, int64_t more) {
        q.rows = r, q.cols = c, q.ld = up(c, 16) + more, q.blocks = blocks;
        const int64_t lines = blocks == FSDP_Q8_ROWS ? down(c) : down(r);
        const int64_t length = blocks == FSDP_Q8_ROWS ? r : blocks == FSDP_Q8_COLS ? c : down(c);
        q.pitch = up(length, 4);
        q.codes = get(at + (r > 0 ? (r - 1) * q.ld + c : 0)) + at;
        q.scales = get(lines > 0 ? (lines - 1) * q.pitch + length : 0);
    }
    uint8_t *get(int64_t n) {
        void *p = nullptr;
        if (posix_memalign(&p, 256, n > 0 ? n : 1) != 0) std::abort();
        held.push_back(p);
        return static_cast<uint8_t *>(p);
    }
    ~Mat() {
        for (void *p : held) std::free(p);
    }
    Mat(const Mat &) = delete;
};

// The linear steps in exactly the memory that they ask for, with the weight and the
// checkpoint at every alignment: the copies of operands, the quantised ones and the
// stretches' sums of each product lie inside it.
void linear(int64_t tokens, int64_t out, int64_t in, int32_t format) {
    for (int where = 0; where < 9; ++where) {
        const int64_t at[3] = {0, 1, 16}, more[3] = {0, 5, 16};
        Mat w(out, in, FSDP_Q8_TILES, at[where / 3], more[where / 3]);
        Mat saved(tokens, in, FSDP_Q8_COLS, at[where % 3], more[where % 3]);
        int64_t need = 0;
        must(fsdp_q8_linear_workspace(&w.q, tokens, &need) == FSDP_OK, "workspace");
        uint8_t *ws = w.get(need);
        std::vector<uint16_t> x(tokens * in + 1), y(tokens * out + 1), dy(tokens * out + 1),
            dx(tokens * in + 1), dw(out * in + 1);
        must(fsdp_q8_linear_forward(&w.q, x.data(), FSDP_DTYPE_BF16, in, tokens, &saved.q, y.data(),
                                    out, ws, need, nullptr) == FSDP_OK,
             "forward");
        for (int which = 1; which < 4; ++which)
            must(fsdp_q8_linear_backward(&w.q, &saved.q, dy.data(), FSDP_DTYPE_BF16, out, format,
                                         which & 1 ? dx.data() : nullptr, in,
                                         which & 2 ? dw.data() : nullptr, in, ws, need,
                                         nullptr) == FSDP_OK,
                 "backward");
    }
}

// One product in exactly its memory; the tile and the stretches it is cut into.
void product(int64_t m, int64_t n, int64_t k, int ta, int tb, int64_t at, int64_t more) {
    Mat a(ta ? k : m, ta ? m : k, ta ? FSDP_Q8_COLS : FSDP_Q8_ROWS, at, more);
    Mat b(tb ? n : k, tb ? k : n, FSDP_Q8_TILES, at, more);
    int64_t need = 0;
    int32_t tile = -1, split = 0;
    must(fsdp_q8_product_workspace(&a.q, ta, &b.q, tb, &need) == FSDP_OK, "workspace");
    must(fsdp_q8_product_cut(&a.q, ta, &b.q, tb, &tile, &split) == FSDP_OK, "cut");
    must(tile == 256 || tile == 128 || tile == 64 || (tile == 0 && m <= 32 && !ta && tb), "tile");
    must(split >= 1 && split <= 16 && (split == 1 || 2 * split * 128 <= up(k, 128)), "split");
    const int64_t copies = up(up(a.q.cols, 16) * a.q.rows, 256) + up(up(b.q.cols, 16) * b.q.rows, 256);
    must(need >= (split > 1 ? 4 * m * n * split : 0), "the stretches' sums");
    must(need <= (split > 1 ? 4 * m * n * split : 0) + copies, "no more");
    if (at == 1) must(need >= copies, "the copies of both operands");
    std::vector<uint16_t> out(m * n + 1);
    must(fsdp_q8_product(&a.q, ta, &b.q, tb, out.data(), n, a.get(need), need, nullptr) == FSDP_OK,
         "product");
}

// Matrices side by side in the same rows share no byte; those that do are refused.
void side_by_side() {
    const int64_t rows = 50, cols = 64, ld = 160;
    std::vector<uint16_t> wide(rows * ld + 64);
    const uint16_t *x = wide.data();
    uint16_t *right = wide.data() + 64;
    Mat q(rows, cols, FSDP_Q8_ROWS, 0, 0), s(rows, cols, FSDP_Q8_COLS, 0, 0);
    Mat w(96, cols, FSDP_Q8_TILES, 0, 0), v(cols, cols, FSDP_Q8_TILES, 0, 0);
    int64_t need = 0;
    must(fsdp_q8_linear_workspace(&w.q, rows, &need) == FSDP_OK, "workspace");
    uint8_t *ws = w.get(need);
    must(fsdp_q8_linear_forward(&w.q, x, FSDP_DTYPE_BF16, ld, rows, &s.q, right, ld, ws, need,
                                nullptr) == FSDP_OK,
         "y to the right of x");
    must(fsdp_q8_linear_backward(&w.q, &s.q, right, FSDP_DTYPE_BF16, ld, FSDP_Q8_E4M3, wide.data(), ld,
                                 nullptr, 0, ws, need, nullptr) == FSDP_OK,
         "dx to the left of dy");
    must(fsdp_q8_linear_forward(&w.q, x, FSDP_DTYPE_BF16, ld, rows, nullptr, right - 1, ld, ws, need,
                                nullptr) == FSDP_E_INVAL,
         "one element shared");
    must(fsdp_q8_linear_forward(&w.q, x, FSDP_DTYPE_BF16, ld, rows, nullptr, right + 1, ld, ws, need,
                                nullptr) == FSDP_E_INVAL,
         "one element of the next row shared");
    must(fsdp_q8_linear_forward(&w.q, x, FSDP_DTYPE_BF16, ld, rows, nullptr, right, ld + 1, ws, need,
                                nullptr) == FSDP_E_INVAL,
         "rows of other lengths");
    // codes of two matrices in the same rows, and of one in the columns it is read from
    Mat two(rows, 2 * cols, FSDP_Q8_ROWS, 0, 0);
    q.q.codes = two.q.codes, s.q.codes = two.q.codes + cols;
    q.q.ld = s.q.ld = two.q.ld;
    must(fsdp_q8_quantize(x, FSDP_DTYPE_BF16, ld, &q.q, &s.q, nullptr) == FSDP_OK, "codes side by side");
    s.q.codes -= 1;
    must(fsdp_q8_quantize(x, FSDP_DTYPE_BF16, ld, &q.q, &s.q, nullptr) == FSDP_E_INVAL, "codes shared");
}

}  // namespace

int main() {
    side_by_side();
    for (int32_t f : {FSDP_Q8_E4M3, FSDP_Q8_E5M2}) {
        linear(70, 260, 515, f);
        linear(1, 1, 1, f);
        linear(300, 128, 256, f);
        linear(0, 40, 50, f);
        linear(1100, 100, 36, f);
        linear(3000, 64, 48, f);
    }
    for (int form = 0; form < 3; ++form)
        for (int odd = 0; odd < 2; ++odd) {
            product(1, 1, 1, form == 2, form == 0, odd, 5 * odd);
            product(32, 500, 300, form == 2, form == 0, odd, 5 * odd);
            product(33, 500, 3000, form == 2, form == 0, odd, 5 * odd);
            product(256, 250, 9000, form == 2, form == 0, odd, 5 * odd);
            product(2000, 1030, 260, form == 2, form == 0, odd, 5 * odd);
            product(3520, 5824, 130, form == 2, form == 0, odd, 5 * odd);
        }
    bind_again();
    out_of_memory();
    std::printf("ALL OK\n");
    return 0;
}
