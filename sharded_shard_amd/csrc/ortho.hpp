// Records and launchers of the orthogonalisation (Newton-Schulz products).
//
// Per matrix the workspace holds, for m = the smaller and n = the larger side
// padded to mp and np (multiples of kOrthoPad, padding zero), X^T as fp16 high
// and low parts ([np][mp]; the high part twice, read and written by turns) and
// the m x m products A and B in fp16.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

namespace fsdp {

constexpr int32_t kOrthoPad = 128;
// at most this many partial sums of squares per matrix
constexpr int32_t kOrthoParts = 256;
// elements per partial sum: at least this many
constexpr int64_t kOrthoPartMin = 16384;

// Per matrix, read on the device; offsets are bytes into the workspace.
struct OrthoMat {
    const void *in;      // [rows, cols] bf16 or fp32
    uint16_t *out;       // [rows, cols] bf16
    int64_t t[2], lo;    // X^T: high parts, low part
    int64_t a, b;        // A, B
    int64_t parts;       // partial sums of squares (double), n_parts of them
    int64_t scal;        // float[4], see OrthoScal
    int32_t rows, cols;
    int32_t m, n, mp, np;
    int32_t n_parts, wide;  // wide: rows <= cols, X = U; else X = U^T
};

// What one init pass leaves for the products: the true X is phi0 times the
// stored one before the first iteration and phi times it after; rho = phi0/phi.
struct OrthoScal {
    float phi0, phi, rho, rsv;
};

struct OrthoTile {
    int32_t mat;
    int32_t ti, tj;
    int32_t rsv;
};

struct OrthoCoef {
    float a, b, c;
};

// Partial sums of squares; tiles: (matrix, part).
hipError_t launch_ortho_norm(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             bool f32, hipStream_t st);
// The scaled X^T and the scalars; tiles: 64 x 64 pieces of [np][mp].  growth:
// log2 of the most that the iterations can magnify a singular value.
hipError_t launch_ortho_init(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             bool f32, double eps, int32_t growth, hipStream_t st);
// A = X X^T, tiles (ti >= tj) of the lower triangle; src: which high part is read.
hipError_t launch_ortho_gram(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             int32_t src, bool first, hipStream_t st);
// B = b A + c A A, tiles of the lower triangle
hipError_t launch_ortho_poly(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             OrthoCoef c, hipStream_t st);
// X^T = a X^T + X^T B into the other high part and the low part, or with last
// into out; tiles (ti of mp, tj of np)
hipError_t launch_ortho_apply(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                              int32_t src, bool first, bool last, OrthoCoef c, hipStream_t st);

}  // namespace fsdp
