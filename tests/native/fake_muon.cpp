// Stand-ins for the launchers of the Muon calls and of the orthogonalisation,
// for the host sanitizer build.  Each walks the tables that the host code
// uploaded and touches the first and last byte of every range a kernel would
// read or write, in the caller's tensors and in the workspace, so that
// AddressSanitizer reports what reaches outside; tiles are recorded for the
// harness, which checks that they cover their matrices exactly once.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <vector>

#include "../../sharded_shard_amd/csrc/muon.hpp"
#include "../../sharded_shard_amd/csrc/ortho.hpp"
#include "muon_harness.hpp"

namespace harness {
std::vector<Launch> ortho;
std::vector<Written> muon;
}  // namespace harness

namespace {

void touch(const void *base, int64_t off, int64_t bytes) {
    if (bytes <= 0) return;
    volatile char a = static_cast<const char *>(base)[off];
    volatile char b = static_cast<const char *>(base)[off + bytes - 1];
    (void)a;
    (void)b;
}

void wrote(const void *base, int64_t off, int64_t len, int64_t esize) {
    touch(base, off * esize, len * esize);
    if (len > 0) harness::muon.push_back({base, off, len});
}

}  // namespace

namespace fsdp {

hipError_t launch_muon_momentum(const PackTile *tiles, int64_t n, const DevEntry *ents,
                                uint16_t *ag_in, const float *, bool, hipStream_t) {
    for (int64_t i = 0; i < n; ++i) {
        const PackTile &t = tiles[i];
        touch(ents[t.entry].grad, t.src * 4, t.valid * 4);
        wrote(ents[t.entry].exp_avg, t.src, t.valid, 4);
        wrote(ag_in, t.dst, t.len, 2);
    }
    return hipSuccess;
}

hipError_t launch_muon_reduce_momentum(const PackTile *tiles, int64_t n, const DevEntry *ents,
                                       const uint16_t *rs_in, uint16_t *ag_in, int64_t S, int32_t N,
                                       const float *, bool, bool, hipStream_t) {
    for (int64_t i = 0; i < n; ++i) {
        const PackTile &t = tiles[i];
        for (int32_t j = 0; j < N; ++j) touch(rs_in, (j * S + t.dst) * 2, t.valid * 2);
        wrote(ents[t.entry].exp_avg, t.src, t.valid, 4);
        wrote(ag_in, t.dst, t.len, 2);
    }
    return hipSuccess;
}

hipError_t launch_muon_update(const PackTile *tiles, int64_t n, const DevEntry *ents,
                              const int64_t *own, const uint16_t *upd, uint16_t *ag_in,
                              const float *scales, const float *, hipStream_t) {
    for (int64_t i = 0; i < n; ++i) {
        const PackTile &t = tiles[i];
        if (upd != nullptr) touch(upd, t.dst * 2, t.valid * 2);
        else touch(ents[t.entry].full, (own[t.entry] + t.src) * 2, t.valid * 2);
        if (scales != nullptr) touch(scales, t.entry * 4, 4);
        wrote(ents[t.entry].master, t.src, t.valid, 4);
        if (ag_in != nullptr) wrote(ag_in, t.dst, t.len, 2);
    }
    return hipSuccess;
}

namespace {

hipError_t record(int what, int32_t tile, const OrthoTile *tiles, int64_t n, int32_t split = 1) {
    harness::ortho.push_back({what, tile, split, std::vector<OrthoTile>(tiles, tiles + n)});
    return hipSuccess;
}

void touch_in(const OrthoMat &M, bool f32) {
    const int64_t n = static_cast<int64_t>(M.rows) * M.cols;
    touch(M.in, 0, n * (f32 ? 4 : 2));
}

}  // namespace

hipError_t launch_ortho_norm(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             bool f32, hipStream_t) {
    for (int64_t i = 0; i < n; ++i) {
        touch_in(mats[tiles[i].mat], f32);
        touch(ws, mats[tiles[i].mat].parts + tiles[i].ti * 8, 8);
    }
    return record(harness::kNorm, 0, tiles, n);
}

hipError_t launch_ortho_init(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             bool f32, double, int32_t, hipStream_t) {
    for (int64_t i = 0; i < n; ++i) {
        const OrthoMat &M = mats[tiles[i].mat];
        touch_in(M, f32);
        const int64_t x = static_cast<int64_t>(M.np) * M.mp * 2;
        for (int64_t at : {M.t[0], M.t[1], M.lo}) touch(ws, at, x);
        touch(ws, M.scal, sizeof(OrthoScal));
    }
    // each piece that a block lays out, as a tile of its own
    std::vector<OrthoTile> pieces;
    for (int64_t i = 0; i < n; ++i)
        for (int32_t k = 0; k < tiles[i].part; ++k)
            pieces.push_back({tiles[i].mat, tiles[i].ti, tiles[i].tj + k, 0});
    return record(harness::kInit, 64, pieces.data(), static_cast<int64_t>(pieces.size()));
}

hipError_t launch_ortho_small(int32_t mp, const OrthoTile *tiles, int64_t n, const OrthoMat *mats,
                              void *ws, bool f32, int32_t mode, int32_t step, int32_t n_steps,
                              const OrthoCoef *coefs, double, int32_t, hipStream_t) {
    touch(coefs, 0, n_steps * sizeof(OrthoCoef));
    const int64_t part = static_cast<int64_t>(small_part(mp)) * 16;
    for (int64_t i = 0; i < n; ++i) {
        const OrthoMat &M = mats[tiles[i].mat];
        if (mode == kSmallAll || mode == kSmallStart) touch_in(M, f32);
        if (mode == kSmallAll || mode == kSmallLast)
            touch(M.out, 0, static_cast<int64_t>(M.rows) * M.cols * 2);
        if (mode == kSmallAll) continue;
        const int64_t image = static_cast<int64_t>(small_slab(mp)) * mp * 4;
        touch(ws, M.t[0] + tiles[i].ti * image, image);
        touch(ws, M.scal, sizeof(OrthoScal));
        if (mode == kSmallStart) touch(ws, M.parts, M.n_parts * 8);
        else touch(ws, (step & 1) ? M.b : M.a, M.n_sums * part);
        if (mode != kSmallLast)
            touch(ws, (((mode == kSmallStart ? 0 : step + 1) & 1) ? M.b : M.a) + tiles[i].ti * part,
                  part);
    }
    return record(harness::kSmall + mode, mp, tiles, n);
}

hipError_t launch_ortho_sums(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             int32_t step, hipStream_t) {
    for (int64_t i = 0; i < n; ++i) {
        const OrthoMat &M = mats[tiles[i].mat];
        const int64_t part = static_cast<int64_t>(small_part(M.mp)) * 16;
        for (int64_t k = 0; k < tiles[i].tj; ++k)
            touch(ws, ((step & 1) ? M.b : M.a) + k * part + tiles[i].ti * 4096, 4096);
    }
    return record(harness::kSums, 0, tiles, n);
}

hipError_t launch_ortho_gram(int32_t tile, const OrthoTile *tiles, int64_t n, const OrthoTile *join,
                             int64_t n_join, int32_t split, const OrthoMat *mats, void *ws, int32_t,
                             bool, hipStream_t) {
    for (int64_t i = 0; i < n; ++i) {
        const OrthoMat &M = mats[tiles[i].mat];
        touch(ws, M.a, static_cast<int64_t>(M.mp) * M.mp * 2);
        if (split > 1)
            touch(ws, M.sums + static_cast<int64_t>(tiles[i].part) * tile * tile * 4,
                  static_cast<int64_t>(tile) * tile * 4);
    }
    if (split > 1) record(harness::kJoin, tile, join, n_join, split);
    return record(harness::kGram, tile, tiles, n, split);
}

hipError_t launch_ortho_poly(int32_t tile, const OrthoTile *tiles, int64_t n, const OrthoMat *mats,
                             void *ws, OrthoCoef, hipStream_t) {
    for (int64_t i = 0; i < n; ++i)
        touch(ws, mats[tiles[i].mat].b, static_cast<int64_t>(mats[tiles[i].mat].mp) *
                                            mats[tiles[i].mat].mp * 2);
    return record(harness::kPoly, tile, tiles, n);
}

hipError_t launch_ortho_apply(int32_t tile, const OrthoTile *tiles, int64_t n,
                              const OrthoMat *mats, void *, int32_t, bool, bool, bool last,
                              OrthoCoef, hipStream_t) {
    for (int64_t i = 0; last && i < n; ++i) {
        const OrthoMat &M = mats[tiles[i].mat];
        touch(M.out, 0, static_cast<int64_t>(M.rows) * M.cols * 2);
    }
    return record(last ? harness::kLast : harness::kApply, tile, tiles, n);
}

}  // namespace fsdp
