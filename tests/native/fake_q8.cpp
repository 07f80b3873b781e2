// Stand-ins for the launchers of the 8-bit matrices, for the host sanitizer build.
// Each touches the first and last byte of every range that a kernel would read or
// write, so that AddressSanitizer reports what reaches outside; the cells of the
// block scales write their bytes, which the harness counts.
#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "../../sharded_shard_amd/csrc/q8.hpp"
#include "q8_harness.hpp"

namespace harness {
int q8_launches = 0;
}

namespace {

void touch(const void *base, int64_t bytes) {
    if (bytes <= 0) return;
    volatile char a = static_cast<const char *>(base)[0];
    volatile char b = static_cast<const char *>(base)[bytes - 1];
    (void)a;
    (void)b;
}

int64_t down(int64_t n) { return (n + 127) / 128; }

void touch(const fsdp::Q8Mat &m) {
    if (m.rows == 0 || m.cols == 0) return;
    touch(m.codes, (m.rows - 1) * m.ld + m.cols);
    if (m.blocks == FSDP_Q8_ROWS) touch(m.scales, (down(m.cols) - 1) * m.pitch + m.rows);
    if (m.blocks == FSDP_Q8_COLS) touch(m.scales, (down(m.rows) - 1) * m.pitch + m.cols);
    if (m.blocks == FSDP_Q8_TILES) touch(m.scales, (down(m.rows) - 1) * m.pitch + down(m.cols));
}

}  // namespace

namespace fsdp {

hipError_t launch_q8_quantize(const void *x, bool f32, int64_t ldx, const Q8Mat &a, const Q8Mat *b,
                              hipStream_t) {
    ++harness::q8_launches;
    if (a.rows > 0 && a.cols > 0) touch(x, ((a.rows - 1) * ldx + a.cols) * (f32 ? 4 : 2));
    touch(a);
    if (b != nullptr) touch(*b);
    return hipSuccess;
}

hipError_t launch_q8_dequantize(const Q8Mat &q, void *out, bool f32, int64_t ldo, hipStream_t) {
    ++harness::q8_launches;
    touch(q);
    if (q.rows > 0 && q.cols > 0) touch(out, ((q.rows - 1) * ldo + q.cols) * (f32 ? 4 : 2));
    return hipSuccess;
}

// Some workspace for every product, whatever its sizes.
Q8Cut q8_cut(const Q8Mat &a, bool ta, const Q8Mat &b, bool tb) {
    Q8Cut c{};
    c.split = 2;
    c.bytes_a = a.rows * 16;
    c.bytes_b = b.cols * 16;
    c.bytes_sums = int64_t{8} * (ta ? a.cols : a.rows) * (tb ? b.rows : b.cols);
    return c;
}

hipError_t launch_q8_product(const Q8Mat &a, bool ta, const Q8Mat &b, bool tb, uint16_t *out,
                             int64_t ldo, const Q8Cut &cut, void *ws, hipStream_t) {
    ++harness::q8_launches;
    touch(a);
    touch(b);
    const int64_t M = ta ? a.cols : a.rows, N = tb ? b.rows : b.cols;
    if (M > 0 && N > 0) touch(out, ((M - 1) * ldo + N) * 2);
    touch(ws, cut.bytes_a + cut.bytes_b + cut.bytes_sums);
    return hipSuccess;
}

hipError_t launch_block_scales(const BlockCell *cells, int64_t n, const BlockEntry *blocks,
                               const DevEntry *ents, uint8_t *scales, hipStream_t) {
    ++harness::q8_launches;
    for (int64_t k = 0; k < n; ++k) {
        const BlockCell &c = cells[k];
        if (c.entry < 0) {
            for (int32_t i = 0; i < c.rows; ++i) ++scales[c.at + i];
            continue;
        }
        const int64_t width = blocks[c.entry].cols;
        const int64_t cols = width - c.col < 128 ? width - c.col : 128;
        const float *p = ents[c.entry].master + c.row * width + c.col;
        touch(p, ((c.rows - 1) * width + cols) * 4);
        scales[c.at] += 2;
    }
    return hipSuccess;
}

hipError_t launch_pack_fp8_blocks(const PackTile *tiles, int64_t n, const BlockEntry *blocks,
                                  const DevEntry *ents, uint8_t *ag_in, const uint8_t *scales,
                                  hipStream_t) {
    ++harness::q8_launches;
    for (int64_t i = 0; i < n; ++i) {
        const PackTile &t = tiles[i];
        touch(ents[t.entry].master + t.src, t.valid * 4);
        touch(ag_in + t.dst, t.len);
        if (t.valid == 0) continue;
        const BlockEntry &b = blocks[t.entry];
        for (int64_t e : {t.src, t.src + t.valid - 1})
            touch(scales + b.at + (b.row_begin + e / b.cols) / 128 * down(b.cols) + e % b.cols / 128, 1);
    }
    return hipSuccess;
}

}  // namespace fsdp
