// 8-bit matrices with a power of two for each block of 128: what the C ABI
// checks (q8.cpp) hand to the kernels (q8.hip, q8_product.hip).  Each launcher
// enqueues on `st` and returns hipGetLastError(); callers have checked every
// argument before.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <vector>

#include "plan.hpp"

namespace fsdp {

// Rows and columns of a matrix, and its leading dimension, at most this: a
// 256-row tile's offsets then fit the 32 bits of a buffer load.
constexpr int64_t kQ8MaxSide = int64_t{1} << 22;

// a block's sides
constexpr int64_t kQ8Block = 128;

// One matrix in 8 bits, as the kernels read and write it.
struct Q8Mat {
    uint8_t *codes;
    uint8_t *scales;
    const float *divisor;   // or null: 1
    int64_t ld, pitch;
    int32_t rows, cols;
    int32_t format;         // FSDP_Q8_E4M3, FSDP_Q8_E5M2
    int32_t blocks;         // FSDP_Q8_TENSOR ... FSDP_Q8_TILES
};

// x [rows, cols] into `a`, and into `b` where it is not null (one of the two
// along rows, the other along columns)
hipError_t launch_q8_quantize(const void *x, bool f32, int64_t ldx, const Q8Mat &a, const Q8Mat *b,
                              hipStream_t st);
hipError_t launch_q8_dequantize(const Q8Mat &q, void *out, bool f32, int64_t ldo, hipStream_t st);

// One block's part on this rank: rows [row, row + rows) of the shard and up to
// 128 columns from `col`; its scale is byte `at`.  With entry -1: the `rows`
// bytes from `at` are of blocks that this rank holds nothing of.
struct BlockCell {
    int64_t row, col, at;
    int32_t entry, rows;
};
static_assert(sizeof(BlockCell) == 32, "BlockCell layout");

// A parameter's blocks: `cols` columns, its shard's first row in the full
// matrix, and the byte of its first block.
struct BlockEntry {
    int64_t cols, row_begin, at;
};

struct Blocks {
    std::vector<BlockEntry> entries;
    std::vector<BlockCell> cells;
    int64_t total = 0;      // bytes of all parameters' scales
};

// Blocks of the full matrices of a layout, and the cells of its rank.
inline Blocks blocks_of(const Layout &L) {
    constexpr int64_t kMost = int64_t{1} << 30;     // bytes a cell of entry -1
    Blocks b;
    for (size_t i = 0; i < L.entries.size(); ++i) {
        const fsdp_shard_entry_t &e = L.entries[i];
        const int64_t across = (e.cols + kQ8Block - 1) / kQ8Block;
        const int64_t down = (e.rows + kQ8Block - 1) / kQ8Block, at = b.total;
        b.entries.push_back({e.cols, e.row_begin, at});
        b.total += across * down;
        const int64_t first = e.local_rows > 0 ? e.row_begin / kQ8Block : down;
        const int64_t end = e.local_rows > 0
                                ? (e.row_begin + e.local_rows + kQ8Block - 1) / kQ8Block
                                : down;
        auto none = [&](int64_t from, int64_t to) {
            for (; from < to; from += kMost)
                b.cells.push_back({0, 0, from, -1,
                                   static_cast<int32_t>(to - from < kMost ? to - from : kMost)});
        };
        none(at, at + first * across);
        for (int64_t r = first; r < end; ++r) {
            const int64_t lo = r * kQ8Block > e.row_begin ? r * kQ8Block : e.row_begin;
            const int64_t last = e.row_begin + e.local_rows;
            const int64_t hi = (r + 1) * kQ8Block < last ? (r + 1) * kQ8Block : last;
            for (int64_t c = 0; c < across; ++c)
                b.cells.push_back({lo - e.row_begin, c * kQ8Block, at + r * across + c,
                                   static_cast<int32_t>(i), static_cast<int32_t>(hi - lo)});
        }
        none(at + end * across, at + down * across);
    }
    return b;
}

// the scales of this rank's part of every block, zeros for the others'
hipError_t launch_block_scales(const BlockCell *cells, int64_t n, const BlockEntry *blocks,
                               const DevEntry *ents, uint8_t *scales, hipStream_t st);
hipError_t launch_pack_fp8_blocks(const PackTile *tiles, int64_t n, const BlockEntry *blocks,
                                  const DevEntry *ents, uint8_t *ag_in, const uint8_t *scales,
                                  hipStream_t st);

// Sides of the results a block makes, by Q8Cut::tile; the last is for up to 32 rows of x W^T,
// whose sums eight waves of a block share.
constexpr int32_t kQ8TileSide[4] = {256, 128, 64, 0};

// How a product is cut up, by its sizes, alignment and strides alone (q8_cut.cpp).
struct Q8Cut {
    int32_t tile;           // index of the tile shape
    int32_t split;          // stretches of the sum, joined by a second launch
    int64_t bytes_a, bytes_b, bytes_sums;   // workspace: aligned copies of operands, the stretches' sums
};
Q8Cut q8_cut(const Q8Mat &a, bool ta, const Q8Mat &b, bool tb);

// out [M, N] bf16 = op(a) op(b)
hipError_t launch_q8_product(const Q8Mat &a, bool ta, const Q8Mat &b, bool tb, uint16_t *out,
                             int64_t ldo, const Q8Cut &cut, void *ws, hipStream_t st);

}  // namespace fsdp
