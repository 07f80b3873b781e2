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

}  // namespace

int main() {
    bind_again();
    out_of_memory();
    std::printf("ALL OK\n");
    return 0;
}
