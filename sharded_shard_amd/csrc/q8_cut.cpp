// How the products of 8-bit matrices are cut up: tile, stretches of the sum, workspace.
#include <cstdint>

#include "q8.hpp"

namespace fsdp {

namespace {

// Microseconds of a product by tiles of one size with its sum in `split` stretches, as
// measured on MI355X: a step takes a block at least `alone`, and the blocks of a CU
// together `each` a block; a launch 3 (with its first loads and its results); joined
// stretches a second launch, and their fp32 sums written and read at 4 TB/s.  Over 45
// products (64 to 14336 rows, all three forms) the choice takes 1.7% more than the best of
// all tiles and stretches on average and 14% at worst (1024 x 4096 x 14336: 81 us for 71).
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

// The same of up to 32 rows of x W^T, for which a block of the path for few rows has 16
// columns and each of its waves every eighth step; 32 columns beyond 4096, one block a CU.
// Where there are many turns of the CUs, or waves have many steps, tiles with the sum in
// stretches are faster: they read b at 6.2 TB/s, this path at 4.7.  A launch of tiles
// counts 5 here.  Over 435 products (64 to 57344 columns, sums of 128 to 28672) the choice
// takes 1.8% more than the better of the two on average, where this path for all takes 12%
// (4% and 14% in a run after the one that gave the constants):
// one row by 4096 x 4096 5.4 us and 9.6 by tiles, 32 rows 8.8 and 10.7; one row by 14336 x
// 4096 13.4 and 15.8, 32 rows 19.5 and 17.1; by 28672 x 8192 46 and 38, 32 rows 64 and 38.
double few_cost(int64_t M, int64_t N, int64_t K, int steps) {
    const bool wide = N > 4096, more = M > 16;
    const double turns = static_cast<double>((N + (wide ? 8191 : 4095)) / (wide ? 8192 : 4096));
    const double step = more ? (wide ? 2.0 : 1.2) : (wide ? 1.3 : 0.6);
    const double us = turns * static_cast<double>((steps + 7) / 8) * step;
    const double read = static_cast<double>(N) * static_cast<double>(K) / 4.7e6;
    return 3.6 + (us > read ? us : read);
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
    double best = 0.0;
    for (int t = 0; t < 3; ++t)
        // stretches of two steps and more
        for (int split = 1; split == 1 || (split <= 16 && split * 2 <= steps); split *= 2) {
            const double us = cost(kTiles[t], kQ8TileSide[t], M, N, steps, split);
            if ((t == 0 && split == 1) || us < best) best = us, c.tile = t, c.split = split;
        }
    if (!ta && tb && M <= 32) {
        const double read = 5.0 + static_cast<double>(N) * static_cast<double>(K) / 6.2e6 +
                            (c.split > 1 ? 3.0 : 0.0);
        if (few_cost(M, N, K, steps) < (best + 2.0 > read ? best + 2.0 : read)) c.tile = 3, c.split = 1;
    }
    // rows along the sum that end inside 16 bytes are copied too, with zeros after them
    c.bytes_a = aligned(a) && (ta || (a.cols & 15) == 0) ? 0 : round256(round16(a.cols) * a.rows);
    c.bytes_b = aligned(b) && (!tb || (b.cols & 15) == 0) ? 0 : round256(round16(b.cols) * b.rows);
    c.bytes_sums = c.split == 1 ? 0 : int64_t{4} * M * N * c.split;
    return c;
}

}  // namespace fsdp
