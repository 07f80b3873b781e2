// Host sanitizer harness of orthogonalisation plans whose products take operands
// of two parts: the workspace's regions are inside it and apart from each other,
// launches ask for the two-part kernels, tiles cover their matrices, and what the
// choice of products refuses.  Against a host-memory HIP (fake_hip.cpp), with
// launch stand-ins of its own.  Prints "ALL OK" when every check passed.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <set>
#include <string>
#include <utility>
#include <vector>

#include "../../include/fsdp_shard.h"
#include "../../sharded_shard_amd/csrc/ortho.hpp"

namespace {

int g_failures = 0;
std::string g_name;
const char *g_ws = nullptr;
int64_t g_bytes = 0;
bool g_fine = false, g_f32 = false;
int g_products = 0;                             // product launches of an execution
std::set<std::pair<int64_t, int64_t>> g_regions;    // offset, bytes

void check(bool ok, const std::string &what) {
    if (ok) return;
    ++g_failures;
    std::fprintf(stderr, "FAIL %s, %s: %s\n", g_name.c_str(), what.c_str(), fsdp_last_error());
}

template <typename T>
T *alloc(int64_t n) {
    void *p = nullptr;
    if (n > 0 && posix_memalign(&p, 256, static_cast<size_t>(n) * sizeof(T)) != 0) std::abort();
    return static_cast<T *>(p);
}

void region(int64_t off, int64_t bytes) { g_regions.insert({off, bytes}); }

// What the products of a matrix read and write.
void regions_of(const fsdp::OrthoMat &M) {
    const int64_t x = static_cast<int64_t>(M.np) * M.mp * 2, s = static_cast<int64_t>(M.mp) * M.mp * 2;
    for (int64_t at : {M.t[0], M.t[1], M.lo}) region(at, x);
    for (int64_t at : {M.a, M.b}) region(at, s);
    if (g_fine) {
        region(M.lo2, x);
        for (int64_t at : {M.al, M.bl}) region(at, s);
    }
    region(M.scal, sizeof(fsdp::OrthoScal));
    region(M.parts, M.n_parts * 8);
    check(M.low == (g_f32 ? 1 : 0), "low part of the start");
}

// The side of a product's tiles; fine or not as the plan.
int32_t side_of(int32_t tile) {
    ++g_products;
    check(((tile & fsdp::kTileFine) != 0) == g_fine, "kernels of the plan's products");
    const int32_t side = tile & ~fsdp::kTileFine;
    check(side == 256 || side == 192 || side == 128 || side == 64, "tile side");
    return side;
}

void cover(int32_t side, const fsdp::OrthoTile *tiles, int64_t n, const fsdp::OrthoMat *mats, bool lower,
           int32_t times) {
    std::map<int32_t, std::map<std::pair<int32_t, int32_t>, int32_t>> seen;
    for (int64_t i = 0; i < n; ++i) ++seen[tiles[i].mat][{tiles[i].ti, tiles[i].tj}];
    for (const auto &m : seen) {
        const fsdp::OrthoMat &M = mats[m.first];
        const int32_t a = (M.mp + side - 1) / side, b = (M.np + side - 1) / side;
        bool ok = static_cast<int64_t>(m.second.size()) ==
                  (lower ? static_cast<int64_t>(a) * (a + 1) / 2 : static_cast<int64_t>(a) * b);
        for (const auto &t : m.second)
            ok = ok && t.second == times && t.first.first < a && t.first.second < (lower ? a : b);
        check(ok, "tiles cover once");
    }
}

}  // namespace

namespace fsdp {

hipError_t launch_ortho_norm(const OrthoTile *, int64_t, const OrthoMat *, void *, bool, hipStream_t) {
    return hipSuccess;
}

hipError_t launch_ortho_init(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *, bool,
                             double, int32_t, hipStream_t) {
    for (int64_t i = 0; i < n; ++i) regions_of(mats[tiles[i].mat]);
    return hipSuccess;
}

hipError_t launch_ortho_small(int32_t, const OrthoTile *, int64_t, const OrthoMat *, void *, bool,
                              int32_t, int32_t, int32_t, const OrthoCoef *, double, int32_t,
                              hipStream_t) {
    return hipSuccess;
}

hipError_t launch_ortho_sums(const OrthoTile *, int64_t, const OrthoMat *, void *, int32_t,
                             hipStream_t) {
    return hipSuccess;
}

hipError_t launch_ortho_gram(int32_t tile, const OrthoTile *tiles, int64_t n, const OrthoTile *join,
                             int64_t n_join, int32_t split, const OrthoMat *mats, void *, int32_t,
                             bool, hipStream_t) {
    const int32_t side = side_of(tile);
    cover(side, tiles, n, mats, true, split);
    if (split > 1) {
        cover(side, join, n_join, mats, true, 1);
        if (n > 0) region(mats[tiles[0].mat].sums, n * side * side * 4);
    }
    return hipSuccess;
}

hipError_t launch_ortho_poly(int32_t tile, const OrthoTile *tiles, int64_t n, const OrthoMat *mats,
                             void *, OrthoCoef, hipStream_t) {
    cover(side_of(tile), tiles, n, mats, true, 1);
    return hipSuccess;
}

hipError_t launch_ortho_apply(int32_t tile, const OrthoTile *tiles, int64_t n, const OrthoMat *mats,
                              void *, int32_t, bool first, bool high, bool, OrthoCoef, hipStream_t) {
    check(high == (first && !g_f32), "the first iteration's low part");
    cover(side_of(tile), tiles, n, mats, false, 1);
    return hipSuccess;
}

}  // namespace fsdp

namespace {

const double kNs[9] = {3.4445, -4.775, 2.0315, 3.4445, -4.775, 2.0315, 1.5, -0.5, 0.0};

void run(const std::string &name, const std::vector<int64_t> &rows, const std::vector<int64_t> &cols,
         int32_t products, bool f32) {
    g_name = name + (f32 ? " fp32" : " bf16") + (products == FSDP_ORTHO_FP16X2 ? " fine" : "");
    g_fine = products == FSDP_ORTHO_FP16X2;
    g_f32 = f32;
    const int32_t n = static_cast<int32_t>(rows.size());
    fsdp_ortho_plan *p = nullptr;
    check(fsdp_ortho_plan_create(rows.data(), cols.data(), n, kNs, 3, 1e-7, &p) == FSDP_OK, "create");
    int32_t mats = 0;
    int64_t plain = 0;
    fsdp_ortho_plan_info(p, &mats, &plain);
    // to and fro: the last choice counts, and a refused one changes nothing
    for (int32_t c : std::vector<int32_t>{FSDP_ORTHO_FP16X2, FSDP_ORTHO_FP16, products})
        check(fsdp_ortho_plan_set_products(p, c) == FSDP_OK, "choice");
    check(fsdp_ortho_plan_set_products(p, 2) == FSDP_E_UNSUPPORTED, "unknown choice");
    check(fsdp_ortho_plan_set_products(nullptr, 0) == FSDP_E_INVAL, "null plan");
    check(fsdp_ortho_plan_info(p, &mats, &g_bytes) == FSDP_OK && mats == n, "info");
    check(products == FSDP_ORTHO_FP16 ? g_bytes == plain : g_bytes >= plain, "workspace bytes");
    std::vector<const void *> in;
    std::vector<uint16_t *> out;
    for (int32_t i = 0; i < n; ++i) {
        in.push_back(alloc<char>(rows[i] * cols[i] * (f32 ? 4 : 2)));
        out.push_back(alloc<uint16_t>(rows[i] * cols[i]));
    }
    char *ws = alloc<char>(g_bytes);
    g_ws = ws;
    check(fsdp_ortho_bind(p, in.data(), out.data(), f32 ? FSDP_DTYPE_F32 : FSDP_DTYPE_BF16, nullptr) ==
              FSDP_OK,
          "bind");
    check(fsdp_ortho_plan_set_products(p, FSDP_ORTHO_FP16) == FSDP_E_STATE, "choice after a bind");
    if (g_bytes > 0)
        check(fsdp_ortho_execute(p, ws, g_bytes - 1, nullptr) == FSDP_E_INVAL, "short workspace");
    g_regions.clear();
    g_products = 0;
    check(fsdp_ortho_execute(p, ws, g_bytes, nullptr) == FSDP_OK, "execute");
    int64_t end = 0;
    bool apart = true;
    for (const auto &r : g_regions) {
        apart = apart && r.first >= end;
        end = r.first + r.second;
    }
    check(apart && end <= g_bytes, "regions of the workspace apart and inside");
    bool big = false;
    for (int32_t i = 0; i < n; ++i) big = big || std::min(rows[i], cols[i]) > fsdp::kSmallMax;
    check(g_products == (big ? 9 : 0), "product launches");
    fsdp_ortho_plan_destroy(p);
    for (int32_t i = 0; i < n; ++i) {
        free(const_cast<void *>(in[i]));
        free(out[i]);
    }
    free(ws);
}

}  // namespace

int main() {
    for (int32_t products : {FSDP_ORTHO_FP16, FSDP_ORTHO_FP16X2})
        for (bool f32 : {false, true}) {
            run("just past few rows", {129, 130, 4000}, {129, 4000, 200}, products, f32);
            run("split sums", {1024, 1024}, {8192, 8192}, products, f32);
            run("mixed", {1408, 64, 300, 0, 5}, {2048, 2048, 400, 3, 9}, products, f32);
            run("few rows", {5, 100}, {7, 20000}, products, f32);
        }
    run("none", {}, {}, FSDP_ORTHO_FP16X2, false);
    if (g_failures != 0) return 1;
    std::puts("ALL OK");
    return 0;
}
