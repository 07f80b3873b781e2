// Records and launchers of the orthogonalisation (Newton-Schulz products).
//
// Per matrix the workspace holds, for m = the smaller and n = the larger side
// padded to mp and np (multiples of kOrthoPad, padding zero), X^T as fp16 high
// and low parts ([np][mp]; the high part twice, read and written by turns) and
// the m x m products A and B in fp16; a fine plan has a low part of A and of B too,
// and both parts of X^T twice.  Where m is at most kSmallMax, and X has
// more columns than a block holds, it has the slabs' X^T, high and low, and two
// sets of the slabs' parts of A in fp32.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

namespace fsdp {

constexpr int32_t kOrthoPad = 128;
// at most this many partial sums of squares per matrix (a decoder block's seven:
// 105 us; 256 of them 116)
constexpr int32_t kOrthoParts = 512;
// elements per partial sum: at least this many
constexpr int64_t kOrthoPartMin = 16384;
// 64 x 64 pieces that one block of the start lays out: two 1024 x 8192 matrices 17.4,
// 14.5, 14.1 and 16.7 us with 1, 2, 4 and 8, a decoder block's seven 179, 171, 175, 177
constexpr int32_t kInitPieces = 2;

// Per matrix, read on the device; offsets are bytes into the workspace.
struct OrthoMat {
    const void *in;      // [rows, cols] bf16 or fp32
    uint16_t *out;       // [rows, cols] bf16
    int64_t t[2], lo;    // X^T: high parts, low part
    int64_t a, b;        // A, B
    int64_t lo2, al, bl; // fine plans: the low part's other place, low parts of A and B
    int64_t parts;       // partial sums of squares (double), n_parts of them
    int64_t scal;        // float[4], see OrthoScal
    int64_t sums;        // fp32 parts of split sums, the plan's
    int32_t rows, cols;
    int32_t m, n, mp, np;
    int32_t n_parts, wide;  // wide: rows <= cols, X = U; else X = U^T
    int32_t n_sums, slab;   // few rows: parts of A that every block sums, columns of a slab
    int32_t low, reserved;  // low: the start leaves a low part (fp32 inputs); set by bind
};

// What one init pass leaves for the products: the true X is phi0 times the
// stored one before the first iteration and phi times it after; rho = phi0/phi.
struct OrthoScal {
    float phi0, phi, rho, rsv;
};

struct OrthoTile {
    int32_t mat;
    int32_t ti, tj;
    int32_t part;        // of a split sum: this part's place among all; start: pieces
};

struct OrthoCoef {
    float a, b, c;
};

// Matrices of at most kSmallMax rows (the smaller side): padded to 32, 64 or
// 128 rows, worked on in slabs of so many columns.
constexpr int32_t kSmallMax = 128;
constexpr int32_t small_rows_of(int32_t m) { return m <= 32 ? 32 : m <= 64 ? 64 : 128; }
// fours of a slab's part of X X^T: the upper 32 x 32 blocks of 128 rows, or all
constexpr int32_t small_part(int32_t mp) { return mp == 128 ? 10 * 256 : mp * mp / 4; }
constexpr int32_t small_slab(int32_t mp) { return mp == 128 ? 128 : mp == 64 ? 416 : 896; }
// with 128 rows the work of one block of threads is long: 16 waves (with 8 a
// 128 x 128 matrix took 7 % longer, 32 of 128 x 2048 18 %)
constexpr int32_t small_threads(int32_t mp) { return mp == 128 ? 1024 : 512; }
// What a launch does: all steps (one slab), the start, one step, the last step.
enum { kSmallAll = 0, kSmallStart = 1, kSmallStep = 2, kSmallLast = 3 };

// Threads of a block of a product with tiles of this side: 256 x 256 by eight
// waves and 192 x 192 by twelve, one block a CU; 128 x 128 and 64 x 64 by four,
// two and five blocks a CU.
constexpr int32_t product_threads(int32_t tile) {
    return tile == 256 ? 512 : tile == 192 ? 768 : 256;
}

// Partial sums of squares; tiles: (matrix, part).
hipError_t launch_ortho_norm(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             bool f32, hipStream_t st);
// The scaled X^T (for fp32 inputs the low part too) and the scalars; tiles: 64 x
// 64 pieces of [np][mp], `part` of them from (tj, ti) on.  growth: log2 of the most that the iterations can
// magnify a singular value.
hipError_t launch_ortho_init(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             bool f32, double eps, int32_t growth, hipStream_t st);
// Matrices of few rows, tiles: (matrix, slab), all of mp padded rows.
hipError_t launch_ortho_small(int32_t mp, const OrthoTile *tiles, int64_t n, const OrthoMat *mats,
                              void *ws, bool f32, int32_t mode, int32_t step, int32_t n_steps,
                              const OrthoCoef *coefs, double eps, int32_t growth, hipStream_t st);
// Sums their parts of step's A where every block would have too many to sum;
// tiles: (matrix, 256 x 4 elements of it, number of parts).
hipError_t launch_ortho_sums(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             int32_t step, hipStream_t st);
// The products; tile: 256, 192, 128 or 64 rows and columns of a tile, plus kTileFine
// for operands of two parts; any other is hipErrorInvalidValue.
constexpr int32_t kTileFine = 1 << 12;
// A = X X^T, tiles (ti >= tj) of the lower triangle; src: which high part is
// read.  With split > 1 every tile comes split times (its part its place among
// all parts), and join has each once, with its first part.
hipError_t launch_ortho_gram(int32_t tile, const OrthoTile *tiles, int64_t n,
                             const OrthoTile *join, int64_t n_join, int32_t split,
                             const OrthoMat *mats, void *ws, int32_t src, bool first,
                             hipStream_t st);
// B = b A + c A A, tiles of the lower triangle
hipError_t launch_ortho_poly(int32_t tile, const OrthoTile *tiles, int64_t n, const OrthoMat *mats,
                             void *ws, OrthoCoef c, hipStream_t st);
// X^T = a X^T + X^T B into the other high part and the low part, or with last
// into out; tiles (ti of mp, tj of np); high: there is no low part yet
hipError_t launch_ortho_apply(int32_t tile, const OrthoTile *tiles, int64_t n,
                              const OrthoMat *mats, void *ws, int32_t src, bool first, bool high,
                              bool last, OrthoCoef c, hipStream_t st);

}  // namespace fsdp
