// How the products of 8-bit matrices are cut up: tile, stretches of the sum, workspace.
#include <cstdint>

#include "q8.hpp"

namespace fsdp {

namespace {

// Microseconds of a product by tiles of one size with its sum in `split` stretches, as
// measured on MI355X: a step takes a block at least `alone`, and the blocks of a CU
// together `each` a block; a launch 3 (with its first loads and its results); joined
// stretches a second launch, and their fp32 sums written and read at 4 TB/s.
struct TileCost {
    int per_cu;
    double alone, each;
};
constexpr TileCost kTiles[3] = {{1, 1.25, 1.50}, {2, 0.60, 0.52}, {4, 0.38, 0.21}};   // 256, 128, 64

double cost(const TileCost &t, int64_t side, int64_t M, int64_t N, int steps, int split) {
    const int64_t items = ((M + side - 1) / side) * ((N + side - 1) / side) * split;
    const int64_t full = items / (256 * t.per_cu), rest = items - full * 256 * t.per_cu;
    auto step = [&](int64_t blocks) {
        const double together = t.each * static_cast<double>((blocks + 255) / 256);
        return blocks == 0 ? 0.0 : together > t.alone ? together : t.alone;
    };
    const double each = (steps + split - 1) / split;
    double us = 3.0 + each * (static_cast<double>(full) * step(256 * t.per_cu) + step(rest));
    if (split > 1) us += 3.0 + 8e-6 * static_cast<double>(M) * static_cast<double>(N) * split / 4.0;
    return us;
}

int64_t round16(int64_t x) { return (x + 15) & ~int64_t{15}; }
int64_t round256(int64_t x) { return (x + 255) & ~int64_t{255}; }

bool aligned(const Q8Mat &m) {
    return (reinterpret_cast<uintptr_t>(m.codes) & 15u) == 0 && (m.ld & 15) == 0;
}

}  // namespace

Q8Cut q8_cut(const Q8Mat &a, bool ta, const Q8Mat &b, bool tb) {
    const int64_t M = ta ? a.cols : a.rows, N = tb ? b.rows : b.cols, K = ta ? a.rows : a.cols;
    const int steps = static_cast<int>((K + kQ8Block - 1) / kQ8Block);
    Q8Cut c{};
    c.split = 1;
    // (one row by 14336 x 4096: 12.5 us for 15.2 by tiles of 64; 32 rows 15.8 either way)
    if (!ta && tb && M <= 32) {
        c.tile = 3;
    } else {
        double best = 0.0;
        for (int t = 0; t < 3; ++t)
            // stretches of two steps and more
            for (int split = 1; split == 1 || (split <= 16 && split * 2 <= steps); split *= 2) {
                const double us = cost(kTiles[t], kQ8TileSide[t], M, N, steps, split);
                if ((t == 0 && split == 1) || us < best) best = us, c.tile = t, c.split = split;
            }
    }
    // rows along the sum that end inside 16 bytes are copied too, with zeros after them
    c.bytes_a = aligned(a) && (ta || (a.cols & 15) == 0) ? 0 : round256(round16(a.cols) * a.rows);
    c.bytes_b = aligned(b) && (!tb || (b.cols & 15) == 0) ? 0 : round256(round16(b.cols) * b.rows);
    c.bytes_sums = c.split == 1 ? 0 : int64_t{4} * M * N * c.split;
    return c;
}

}  // namespace fsdp
