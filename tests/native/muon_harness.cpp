// Host sanitizer harness of the Muon calls and of the orthogonalisation plans:
// their host code (argument checks, workspace layout, tiles, device tables) with
// AddressSanitizer and UndefinedBehaviorSanitizer, against a host-memory HIP
// (fake_hip.cpp) and launch stand-ins (fake_muon.cpp).  Every tensor and the
// workspace are exact-size allocations.  Prints "ALL OK" when every check passed.
#include "muon_harness.hpp"

#include <cstdio>
#include <cstdlib>
#include <map>
#include <set>
#include <string>
#include <tuple>
#include <vector>

#include "../../include/fsdp_shard.h"

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

// Each element of [0, n) of base written once.
void check_cover(const void *base, int64_t n, const std::string &what) {
    std::vector<uint8_t> hits(static_cast<size_t>(n), 0);
    bool ok = true;
    for (const harness::Written &w : harness::muon) {
        if (w.base != base) continue;
        for (int64_t i = w.off; i < w.off + w.len; ++i) {
            if (i < 0 || i >= n || hits[i]++) ok = false;
        }
    }
    for (uint8_t h : hits) ok = ok && h == 1;
    check(ok, what + ": not every element written once");
}

void muon(const std::vector<int64_t> &rows, const std::vector<int64_t> &cols, int32_t world,
          int32_t rank, int32_t align) {
    const int32_t n = static_cast<int32_t>(rows.size());
    fsdp_plan *p = nullptr;
    check(fsdp_plan_create(rows.data(), cols.data(), n, world, rank, align, &p) == FSDP_OK, "plan");
    fsdp_plan_info_t info;
    fsdp_plan_info(p, &info);
    std::vector<float *> master, grad, m;
    std::vector<uint16_t *> full;
    std::vector<fsdp_shard_entry_t> ents(n);
    for (auto *v : {&master, &grad, &m}) v->reserve(1);     // an array even of none
    full.reserve(1);
    for (int32_t i = 0; i < n; ++i) {
        fsdp_plan_entry(p, i, &ents[i]);
        master.push_back(alloc<float>(ents[i].valid_numel));
        grad.push_back(alloc<float>(ents[i].valid_numel));
        m.push_back(alloc<float>(ents[i].valid_numel));
        full.push_back(alloc<uint16_t>(rows[i] * cols[i]));
    }
    uint16_t *seg = alloc<uint16_t>(info.S), *upd = alloc<uint16_t>(info.S);
    uint16_t *rs = alloc<uint16_t>(info.S * world);
    float *scales = alloc<float>(n);
    const fsdp_muon_hparams_t hp = {0.02, 0.95, 0.1, 1, 0};
    check(fsdp_muon_momentum(p, seg, &hp, nullptr) == FSDP_E_STATE, "unbound momentum");
    check(fsdp_muon_update(p, upd, seg, scales, &hp, nullptr) == FSDP_E_STATE, "unbound update");
    check(fsdp_bind(p, master.data(), grad.data(), m.data(), nullptr, nullptr, nullptr) == FSDP_OK,
          "bind");
    if (info.S > 0)
        check(fsdp_muon_update(p, nullptr, seg, scales, &hp, nullptr) == FSDP_E_STATE, "no rows bound");
    check(fsdp_bind(p, nullptr, nullptr, nullptr, nullptr, full.data(), nullptr) == FSDP_OK, "bind");
    auto state = [&](const std::vector<float *> &t, const char *what) {
        for (int32_t i = 0; i < n; ++i)
            if (ents[i].valid_numel > 0) check_cover(t[i], ents[i].valid_numel, what);
        if (info.S > 0) check_cover(seg, info.S, std::string(what) + " segment");
        harness::muon.clear();
    };
    check(fsdp_muon_momentum(p, seg, &hp, nullptr) == FSDP_OK, "momentum");
    state(m, "momentum");
    check(fsdp_muon_reduce_momentum(p, rs, seg, &hp, nullptr) == FSDP_OK, "reduce momentum");
    state(m, "reduce momentum");
    check(fsdp_muon_update(p, upd, seg, scales, &hp, nullptr) == FSDP_OK, "update");
    state(master, "update");
    check(fsdp_muon_update(p, nullptr, seg, nullptr, &hp, nullptr) == FSDP_OK, "update from rows");
    state(master, "update from rows");
    check(fsdp_muon_update(p, upd, nullptr, nullptr, &hp, nullptr) == FSDP_OK, "update alone");
    harness::muon.clear();
    setenv("FSDP_FAULT", "launch", 1);
    check(fsdp_muon_momentum(p, seg, &hp, nullptr) == FSDP_E_HIP, "injected fault");
    unsetenv("FSDP_FAULT");
    check(harness::muon.empty(), "nothing launched after a fault");
    fsdp_plan_destroy(p);
    for (int32_t i = 0; i < n; ++i) {
        free(master[i]);
        free(grad[i]);
        free(m[i]);
        free(full[i]);
    }
    free(seg);
    free(upd);
    free(rs);
    free(scales);
}

// The tiles of one launch cover each matrix of `want` (mat -> rows, columns of
// tiles) once, the lower triangle alone with `lower`.
void check_tiles(const harness::Launch &l, const std::map<int32_t, std::pair<int32_t, int32_t>> &want,
                 bool lower, const std::string &what) {
    std::map<std::tuple<int32_t, int32_t, int32_t>, int32_t> seen;
    std::set<int32_t> parts;
    bool ok = true;
    for (const fsdp::OrthoTile &t : l.tiles) {
        auto it = want.find(t.mat);
        ok = ok && it != want.end() && t.ti >= 0 && t.ti < it->second.first && t.tj >= 0 &&
             t.tj < it->second.second && (!lower || t.tj <= t.ti);
        ++seen[{t.mat, t.ti, t.tj}];
        if (l.split > 1) ok = ok && parts.insert(t.part).second;
    }
    size_t total = 0;
    for (const auto &w : want) {
        const size_t a = w.second.first, b = w.second.second;
        total += lower ? a * (a + 1) / 2 : a * b;
    }
    const int32_t times = what.find("join") != std::string::npos ? 1 : l.split;
    for (const auto &s : seen) ok = ok && s.second == times;
    check(ok && seen.size() == total, what + ": tiles do not cover once");
}

void ortho(const std::vector<int64_t> &rows, const std::vector<int64_t> &cols, bool f32,
           const std::string &name) {
    const int32_t n = static_cast<int32_t>(rows.size());
    const int32_t steps = 3;
    const double ns[9] = {3.4445, -4.775, 2.0315, 3.4445, -4.775, 2.0315, 1.5, -0.5, 0.0};
    fsdp_ortho_plan *p = nullptr;
    check(fsdp_ortho_plan_create(rows.data(), cols.data(), n, ns, steps, 1e-7, &p) == FSDP_OK, name);
    int32_t got = 0;
    int64_t bytes = 0;
    check(fsdp_ortho_plan_info(p, &got, &bytes) == FSDP_OK && got == n, name + " info");
    std::vector<const void *> in;
    std::vector<uint16_t *> out;
    std::vector<std::pair<int32_t, int32_t>> sides;     // of the matrices with elements
    for (int32_t i = 0; i < n; ++i) {
        in.push_back(alloc<char>(rows[i] * cols[i] * (f32 ? 4 : 2)));
        out.push_back(alloc<uint16_t>(rows[i] * cols[i]));
        if (rows[i] * cols[i] > 0)
            sides.push_back({static_cast<int32_t>(std::min(rows[i], cols[i])),
                             static_cast<int32_t>(std::max(rows[i], cols[i]))});
    }
    char *ws = alloc<char>(bytes);
    check(fsdp_ortho_execute(p, ws, bytes, nullptr) == FSDP_E_STATE, name + " unbound");
    for (int turn = 0; turn < 2; ++turn)        // binding again replaces the tables
        check(fsdp_ortho_bind(p, in.data(), out.data(), f32 ? FSDP_DTYPE_F32 : FSDP_DTYPE_BF16,
                              nullptr) == FSDP_OK,
              name + " bind");
    if (bytes > 0)
        check(fsdp_ortho_execute(p, ws, bytes - 1, nullptr) == FSDP_E_INVAL, name + " short");
    harness::ortho.clear();
    check(fsdp_ortho_execute(p, ws, bytes, nullptr) == FSDP_OK, name + " execute");
    int64_t counts[16] = {0};
    auto up = [](int32_t x, int32_t a) { return (x + a - 1) / a; };
    for (const harness::Launch &l : harness::ortho) {
        ++counts[l.what];
        std::map<int32_t, std::pair<int32_t, int32_t>> want;
        const bool small = l.what >= harness::kSmall;
        for (size_t k = 0; k < sides.size(); ++k) {
            const int32_t m = sides[k].first, nn = sides[k].second, id = static_cast<int32_t>(k);
            const bool few = m <= fsdp::kSmallMax;
            const int32_t mp = few ? fsdp::small_rows_of(m) : up(m, 128) * 128, np = up(nn, 128) * 128;
            if (few != small) continue;
            if (l.what == harness::kInit) want[id] = {mp / 64, np / 64};
            if (l.what == harness::kGram || l.what == harness::kJoin || l.what == harness::kPoly)
                want[id] = {up(mp, l.tile), up(mp, l.tile)};
            if (l.what == harness::kApply || l.what == harness::kLast)
                want[id] = {up(mp, l.tile), up(np, l.tile)};
            if (l.what == harness::kSmall && l.tile == mp && nn <= fsdp::small_slab(mp))
                want[id] = {1, 1};
        }
        if (l.what == harness::kNorm || l.what == harness::kSums || l.what > harness::kSmall) continue;
        const bool lower = l.what == harness::kGram || l.what == harness::kJoin || l.what == harness::kPoly;
        check_tiles(l, want, lower, name + (l.what == harness::kJoin ? " join" : " launch ") +
                                        std::to_string(l.what));
    }
    bool big = false;
    for (const auto &s : sides) big = big || s.first > fsdp::kSmallMax;
    if (big)
        check(counts[harness::kGram] == steps && counts[harness::kPoly] == steps &&
                  counts[harness::kApply] == steps - 1 && counts[harness::kLast] == 1,
              name + ": launches of the products");
    const int64_t slabs = counts[harness::kSmall + fsdp::kSmallStart];
    check(counts[harness::kSmall + fsdp::kSmallLast] == slabs &&
              counts[harness::kSmall + fsdp::kSmallStep] == slabs * (steps - 1),
          name + ": launches of the slabs");
    setenv("FSDP_FAULT", "launch@2", 1);
    harness::ortho.clear();
    const bool more = fsdp_ortho_execute(p, ws, bytes, nullptr) == FSDP_E_HIP;
    unsetenv("FSDP_FAULT");
    check(!more || harness::ortho.size() <= 2, name + ": nothing launched after a fault");
    fsdp_ortho_plan_destroy(p);
    for (int32_t i = 0; i < n; ++i) {
        free(const_cast<void *>(in[i]));
        free(out[i]);
    }
    free(ws);
}

}  // namespace

int main() {
    for (int32_t align : {1, 8})
        for (int32_t rank : {0, 1, 5}) {
            muon({1000, 77, 1, 64}, {70, 129, 2048, 32}, 6, rank, align);
            muon({5, 0, 1, 13}, {3, 4, 5, 2}, 6, rank, align);
        }
    muon({}, {}, 1, 0, 1);
    for (bool f32 : {false, true}) {
        ortho({5, 0, 300, 7}, {7, 4, 20, 0}, f32, "few rows");
        ortho({1, 3, 100, 128, 50, 33, 2000}, {5000, 100001, 130, 3000, 20000, 897, 60}, f32, "slabs");
        ortho({129, 130, 4000}, {129, 4000, 200}, f32, "just past few rows");
        ortho({1024, 1024}, {8192, 8192}, f32, "split sums");
        ortho({4096}, {4096}, f32, "square");
        ortho({1408, 1408, 2048, 64, 1, 0}, {2048, 2048, 1408, 2048, 2048, 7}, f32, "experts");
    }
    ortho({}, {}, false, "none");
    if (g_failures != 0) return 1;
    std::puts("ALL OK");
    return 0;
}
