// Host sanitizer harness of what orthogonalisation plans refuse and what they
// keep over several binds, against a host-memory HIP (fake_hip.cpp) and launch
// stand-ins (fake_muon.cpp), which touch the first and last byte of every range
// a kernel would.  Every tensor is an exact-size allocation.  Prints "ALL OK"
// when every check passed.
#include <cstdio>
#include <cstdlib>
#include <string>
#include <vector>

#include "../../include/fsdp_shard.h"
#include "muon_harness.hpp"

namespace {

int g_failures = 0;

void check(bool ok, const std::string &what) {
    if (ok) return;
    ++g_failures;
    std::fprintf(stderr, "FAIL %s: %s\n", what.c_str(), fsdp_last_error());
}

template <typename T>
T *alloc(int64_t n) {
    void *p = nullptr;
    if (n > 0 && posix_memalign(&p, 256, static_cast<size_t>(n) * sizeof(T)) != 0) std::abort();
    return static_cast<T *>(p);
}

const double kNs[6] = {3.4445, -4.775, 2.0315, 3.4445, -4.775, 2.0315};

// Executions hold the kernels of the first bind's dtype: no later bind may name
// inputs of another one, and a refused one changes nothing.
void dtype_is_the_first_binds(int32_t first, int64_t rows, int64_t cols) {
    const std::string name = first == FSDP_DTYPE_F32 ? "fp32 first" : "bf16 first";
    const int32_t other = first == FSDP_DTYPE_F32 ? FSDP_DTYPE_BF16 : FSDP_DTYPE_F32;
    const int64_t n = rows * cols;
    fsdp_ortho_plan *p = nullptr;
    check(fsdp_ortho_plan_create(&rows, &cols, 1, kNs, 2, 1e-7, &p) == FSDP_OK, name + " create");
    int32_t mats = 0;
    int64_t bytes = 0;
    check(fsdp_ortho_plan_info(p, &mats, &bytes) == FSDP_OK && mats == 1, name + " info");
    char *ws = alloc<char>(bytes), *half = alloc<char>(2 * n), *full = alloc<char>(4 * n);
    uint16_t *outs[2] = {alloc<uint16_t>(n), alloc<uint16_t>(n)};
    const void *in = first == FSDP_DTYPE_F32 ? full : half;
    const void *in2 = first == FSDP_DTYPE_F32 ? half : full;
    // a bind that is refused sets nothing
    const void *none = nullptr;
    check(fsdp_ortho_bind(p, &none, &outs[0], other, nullptr) == FSDP_E_INVAL, name + " null input");
    check(fsdp_ortho_bind(p, &in, &outs[0], first, nullptr) == FSDP_OK, name + " bind");
    check(fsdp_ortho_bind(p, &in2, &outs[1], other, nullptr) == FSDP_E_STATE, name + " other dtype");
    check(fsdp_ortho_execute(p, ws, bytes, nullptr) == FSDP_OK, name + " still bound");
    check(fsdp_ortho_bind(p, &in, &outs[1], first, nullptr) == FSDP_OK, name + " other memory");
    check(fsdp_ortho_execute(p, ws, bytes, nullptr) == FSDP_OK, name + " execute");
    fsdp_ortho_plan_destroy(p);
    for (void *q : {static_cast<void *>(ws), static_cast<void *>(half), static_cast<void *>(full),
                    static_cast<void *>(outs[0]), static_cast<void *>(outs[1])})
        free(q);
}

}  // namespace

int main() {
    for (int32_t first : {FSDP_DTYPE_BF16, FSDP_DTYPE_F32})
        for (int64_t cols : {33, 2000})
            for (int64_t rows : {20, 200}) dtype_is_the_first_binds(first, rows, cols);
    if (g_failures != 0) return 1;
    std::puts("ALL OK");
    return 0;
}
