// The host code of the 8-bit matrices under AddressSanitizer: device tables and the
// cells of the block scales on ragged layouts, workspaces of the linear steps, against
// exact-size allocations.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <vector>

#include "../../include/fsdp_shard.h"
#include "q8_harness.hpp"

namespace {

void must(bool ok, const char *what) {
    if (ok) return;
    std::printf("FAILED %s: %s\n", what, fsdp_last_error());
    std::exit(1);
}

// Exactly n elements, 256-byte aligned from the front.
template <typename T>
struct Buf {
    T *p;
    explicit Buf(int64_t n) {
        void *q = nullptr;
        if (posix_memalign(&q, 256, n > 0 ? n * sizeof(T) : 1) != 0) std::abort();
        p = static_cast<T *>(q);
    }
    ~Buf() { std::free(p); }
    Buf(const Buf &) = delete;
};

int64_t down(int64_t n) { return (n + 127) / 128; }

struct Mat {
    fsdp_q8_t q{};
    Buf<uint8_t> codes, scales;
    static int64_t lines(int64_t r, int64_t c, int b) {
        return b == FSDP_Q8_ROWS ? down(c) : down(r);
    }
    static int64_t length(int64_t r, int64_t c, int b) {
        return b == FSDP_Q8_ROWS ? r : b == FSDP_Q8_COLS ? c : down(c);
    }
    Mat(int64_t r, int64_t c, int blocks)
        : codes(r > 0 && c > 0 ? (r - 1) * (c + 3) + c : 0),
          scales(r > 0 && c > 0 ? (lines(r, c, blocks) - 1) * ((length(r, c, blocks) + 3) / 4 * 4) +
                                      length(r, c, blocks)
                                : 0) {
        q.codes = codes.p;
        q.scales = scales.p;
        q.rows = r, q.cols = c, q.ld = c + 3;
        q.pitch = (length(r, c, blocks) + 3) / 4 * 4;
        q.blocks = blocks;
    }
};

void copy_in(std::initializer_list<std::pair<int64_t, int64_t>> shapes, int world) {
    std::vector<int64_t> rows, cols;
    for (auto &s : shapes) rows.push_back(s.first), cols.push_back(s.second);
    const int n = static_cast<int>(rows.size());
    for (int align : {1, 8})
        for (int rank = 0; rank < world; ++rank) {
            fsdp_plan *plan = nullptr;
            must(fsdp_plan_create(rows.data(), cols.data(), n, world, rank, align, &plan) == FSDP_OK,
                 "plan");
            std::vector<Buf<float> *> shards;
            std::vector<float *> master;
            fsdp_plan_info_t info;
            fsdp_plan_info(plan, &info);
            for (int i = 0; i < n; ++i) {
                fsdp_shard_entry_t e;
                fsdp_plan_entry(plan, i, &e);
                shards.push_back(new Buf<float>(e.valid_numel));
                master.push_back(shards.back()->p);
            }
            must(fsdp_bind(plan, master.data(), nullptr, nullptr, nullptr, nullptr, nullptr) == FSDP_OK,
                 "bind");
            int64_t at = 0, total = 0;
            must(fsdp_plan_block_scales(plan, 0, &at, &total) == FSDP_OK, "block scales");
            Buf<uint8_t> scales(total), seg(info.S);
            for (int64_t i = 0; i < total; ++i) scales.p[i] = 0;
            must(fsdp_block_scales_shard(plan, scales.p, nullptr) == FSDP_OK, "scales");
            // every byte once: 1 where the rank has nothing of the block, 2 where it has
            for (int i = 0; i < n; ++i) {
                fsdp_shard_entry_t e;
                fsdp_plan_entry(plan, i, &e);
                fsdp_plan_block_scales(plan, i, &at, &total);
                for (int64_t r = 0; r < down(rows[i]); ++r)
                    for (int64_t c = 0; c < down(cols[i]); ++c) {
                        const bool mine = e.local_rows > 0 && r * 128 < e.row_begin + e.local_rows &&
                                          (r + 1) * 128 > e.row_begin;
                        must(scales.p[at + r * down(cols[i]) + c] == (mine ? 2 : 1), "cover");
                    }
            }
            must(fsdp_pack_allgather_fp8_blocks(plan, seg.p, scales.p, nullptr) == FSDP_OK, "pack");
            fsdp_plan_destroy(plan);
            for (auto *b : shards) delete b;
        }
}

void linear(int64_t tokens, int64_t out, int64_t in, int32_t format) {
    Mat w(out, in, FSDP_Q8_TILES), saved(tokens, in, FSDP_Q8_COLS);
    Buf<uint16_t> x(tokens * in), y(tokens * out), dy(tokens * out), dx(tokens * in), dw(out * in);
    int64_t bytes = 0;
    must(fsdp_q8_linear_workspace(&w.q, tokens, &bytes) == FSDP_OK, "workspace");
    Buf<char> ws(bytes);
    must(fsdp_q8_linear_forward(&w.q, x.p, FSDP_DTYPE_BF16, in, tokens, &saved.q, y.p, out, ws.p, bytes,
                                nullptr) == FSDP_OK,
         "forward");
    for (int which = 0; which < 4; ++which)
        must(fsdp_q8_linear_backward(&w.q, &saved.q, dy.p, FSDP_DTYPE_BF16, out, format,
                                     which & 1 ? dx.p : nullptr, in, which & 2 ? dw.p : nullptr, in, ws.p,
                                     bytes, nullptr) == FSDP_OK,
             "backward");
    if (bytes > 0) {
        must(fsdp_q8_linear_forward(&w.q, x.p, FSDP_DTYPE_BF16, in, tokens, nullptr, y.p, out, ws.p,
                                    bytes - 1, nullptr) == FSDP_E_INVAL,
             "a byte less");
    }
    for (int blocks : {FSDP_Q8_ROWS, FSDP_Q8_COLS, FSDP_Q8_TILES}) {
        Mat q(tokens, in, blocks);
        must(fsdp_q8_quantize(x.p, FSDP_DTYPE_BF16, in, &q.q, nullptr, nullptr) == FSDP_OK, "quantize");
        must(fsdp_q8_dequantize(&q.q, dx.p, FSDP_DTYPE_BF16, in, nullptr) == FSDP_OK, "dequantize");
    }
    Mat rows(tokens, in, FSDP_Q8_ROWS);
    must(fsdp_q8_product_workspace(&rows.q, 0, &w.q, 1, &bytes) == FSDP_OK, "product workspace");
    Buf<char> wp(bytes);
    must(fsdp_q8_product(&rows.q, 0, &w.q, 1, y.p, out, wp.p, bytes, nullptr) == FSDP_OK, "product");
    // an injected failure: nothing after it
    setenv("FSDP_FAULT", "launch@2", 1);
    const int before = harness::q8_launches;
    fsdp_q8_linear_workspace(&w.q, tokens, &bytes);
    must(fsdp_q8_linear_backward(&w.q, &saved.q, dy.p, FSDP_DTYPE_BF16, out, format, dx.p, in, dw.p, in,
                                 ws.p, bytes, nullptr) == FSDP_E_HIP,
         "fault");
    must(harness::q8_launches == before + 1, "launches after a fault");
    unsetenv("FSDP_FAULT");
    must(fsdp_q8_dequantize(&rows.q, dx.p, FSDP_DTYPE_BF16, in, nullptr) == FSDP_OK, "after");
}

}  // namespace

int main() {
    copy_in({{32, 16}, {32, 1}, {4, 32}, {4, 1}}, 2);
    copy_in({{1000, 70}, {333, 1}, {77, 129}, {1, 2048}, {1, 1}, {64, 2048}}, 6);
    copy_in({{5, 3}, {0, 4}, {7, 1}, {1, 5}, {13, 2}}, 4);
    copy_in({{300, 1000}, {4096, 33}, {70001, 1}}, 8);
    copy_in({{3, 70001}, {129, 128}, {128, 129}}, 1);
    for (int32_t f : {FSDP_Q8_E4M3, FSDP_Q8_E5M2}) {
        linear(70, 260, 515, f);
        linear(1, 1, 1, f);
        linear(300, 128, 256, f);
        linear(0, 40, 50, f);
    }
    std::printf("ALL OK\n");
    return 0;
}
