// 8-bit matrices with a power of two for each block of 128: from bf16 or fp32,
// back, and the FP8 copy-in of the fp32 shards with such scales.
//
// A block whose largest finite magnitude is a has the smallest s = 2^(byte -
// 127) with a <= fmax s, fmax = 7/8 of a power of two (448 = 0.875 2^9 for
// E4M3, 57344 = 0.875 2^16 for E5M2).  x / s is exact, so a value is rounded
// once, when it becomes a code; the byte grows with a, so the maximum of
// several ranks' bytes is the byte of their maximum; and the matrix
// instructions take the byte as it is.  What is not finite has no part in the
// scale: NaN stays NaN, an infinity is one in E5M2 and NaN in E4M3, so that
// what overflowed before still shows after.
#include "q8.hpp"

#include "device.hpp"

namespace fsdp {

namespace {

// ---------------------------------------------------------------------------
// scales and codes
// ---------------------------------------------------------------------------

// |x|'s bits, 0 where x is not finite
__device__ __forceinline__ uint32_t finite_mag(float x) {
    const uint32_t m = __float_as_uint(x) & 0x7FFFFFFFu;
    return m < 0x7F800000u ? m : 0u;
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The scale's byte for the magnitude with these bits, 2^e (1 + f): fmax s is
// 1.75 2^(byte - 127 + kLog), so a fits from byte = e + 127 - kLog on, or one
// more where 1 + f > 1.75.  Subnormal and zero magnitudes give byte 0.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t mag) {
    constexpr int kLog = FMT == FSDP_Q8_E4M3 ? 8 : 15;
    const int b = static_cast<int>(mag >> 23) - kLog + ((mag & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return static_cast<uint32_t>(b < 0 ? 0 : b);
}

// 2^(127 - byte), what x is multiplied by; 255 is NaN
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
    const uint32_t up = byte < 254u ? (254u - byte) << 23 : 0x400000u;
    return __uint_as_float(byte == 255u ? 0x7FC00000u : up);
}

// 2^(byte - 127)
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x400000u : byte << 23);
}

// Four codes, by the converter (to nearest even).  Finite values that would
// round past fmax, which only a caller's scales can leave, are clamped to it;
// the comparisons keep NaN.
template <int FMT>
__device__ __forceinline__ float clamped(float x) {
    constexpr float kMax = FMT == FSDP_Q8_E4M3 ? 448.0f : 57344.0f;
    // an infinity is no value that a code could stand in for: NaN for E4M3
    if constexpr (FMT == FSDP_Q8_E4M3) x = fabsf(x) == __builtin_inff() ? __builtin_nanf("") : x;
    else if (fabsf(x) == __builtin_inff()) return x;
    return x > kMax ? kMax : (x < -kMax ? -kMax : x);
}

template <int FMT>
__device__ __forceinline__ uint32_t four_codes(float a, float b, float c, float d) {
    int w;
    if constexpr (FMT == FSDP_Q8_E4M3) {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(clamped<FMT>(a), clamped<FMT>(b), 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(clamped<FMT>(c), clamped<FMT>(d), w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(clamped<FMT>(a), clamped<FMT>(b), 0, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(clamped<FMT>(c), clamped<FMT>(d), w, true);
    }
    return static_cast<uint32_t>(w);
}

// ---------------------------------------------------------------------------
// quantise
// ---------------------------------------------------------------------------

// Eight neighbouring values: packed bf16 or fp32.
template <bool kF32>
struct Eight {
    u32x4 w[kF32 ? 2 : 1];
    __device__ __forceinline__ float get(int e) const {
        if constexpr (kF32) return __uint_as_float(w[e >> 2][e & 3]);
        else return e & 1 ? bf16_hi(w[0][e >> 1]) : bf16_lo(w[0][e >> 1]);
    }
};

// n of eight values at element o of x, zeros for the others; vec: one or two
// aligned loads for all eight.
template <bool kF32>
__device__ __forceinline__ Eight<kF32> load_eight(const void *x, int64_t o, int n, bool vec) {
    Eight<kF32> v;
    if (vec && n == 8) {
        if constexpr (kF32) {
            const u32x4 *p = reinterpret_cast<const u32x4 *>(static_cast<const float *>(x) + o);
            v.w[0] = p[0];
            v.w[1] = p[1];
        } else {
            v.w[0] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(x) + o);
        }
        return v;
    }
    if constexpr (kF32) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v.w[e >> 2][e & 3] = e < n ? static_cast<const uint32_t *>(x)[o + e] : 0u;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint16_t *p = static_cast<const uint16_t *>(x) + o + 2 * e;
            const uint32_t lo = 2 * e < n ? p[0] : 0u, hi = 2 * e + 1 < n ? p[1] : 0u;
            v.w[0][e] = lo | hi << 16;
        }
    }
    return v;
}

__device__ __forceinline__ uint32_t lane_max(uint32_t v, int from, int to) {
    for (int d = from; d < to; d <<= 1)
        v = umax(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), d, 64)));
    return v;
}

// n of eight codes at p; vec: one store of all eight
__device__ __forceinline__ void store_eight(uint8_t *p, uint32_t lo, uint32_t hi, int n, bool vec) {
    if (vec && n == 8) {
        *reinterpret_cast<u32x2 *>(p) = u32x2{lo, hi};
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) p[e] = static_cast<uint8_t>((e < 4 ? lo : hi) >> (8 * (e & 3)));
}

enum { kWriteRows = 1, kWriteCols = 2, kWriteTiles = 4 };

// One 128 x 128 block a workgroup, held in registers from the loads to the
// stores: thread (r, c) of 16 x 16 has the eight columns from 8 c of the rows r,
// r + 16, ...  A row's maximum is taken over its 16 neighbouring lanes, a
// column's over the wave's four rows and, through LDS, over the waves.
template <int FMT, bool kF32, int WHAT>
__global__ __launch_bounds__(kBlock) void q8_quantize_kernel(const void *__restrict__ x,
                                                             int64_t ldx, Q8Mat A, Q8Mat B) {
    __shared__ uint32_t part[4][128];
    __shared__ __attribute__((aligned(16))) uint8_t bytes[2][128];
    const int tid = threadIdx.x, r = tid >> 4, c = (tid & 15) * 8, wave = tid >> 6;
    const int row0 = blockIdx.y * 128, col0 = blockIdx.x * 128;
    const int rows = A.rows - row0 < 128 ? A.rows - row0 : 128;
    const int cols = A.cols - col0 < 128 ? A.cols - col0 : 128;
    const int n = cols - c < 0 ? 0 : (cols - c < 8 ? cols - c : 8);
    const bool vec = (lo32(x) & 15u) == 0 && (ldx & (kF32 ? 3 : 7)) == 0;
    const Q8Mat &rm = A, &cm = (WHAT & kWriteRows) && (WHAT & kWriteCols) ? B : A;
    Eight<kF32> v[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int row = r + 16 * p;
        const int64_t o = static_cast<int64_t>(row0 + row) * ldx + col0 + c;
        v[p] = load_eight<kF32>(x, o, row < rows ? n : 0, vec);
    }
    if constexpr (WHAT & kWriteRows) {
        const bool wide = (lo32(rm.codes) & 7u) == 0 && (rm.ld & 7) == 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = umax(m, finite_mag(v[p].get(e)));
            const uint32_t b = scale_byte<FMT>(lane_max(m, 1, 16));
            const float s = inverse_scale(b);
            const int row = r + 16 * p;
            if ((tid & 15) == 0) bytes[0][row] = static_cast<uint8_t>(b);
            if (row < rows)
                store_eight(rm.codes + static_cast<int64_t>(row0 + row) * rm.ld + col0 + c,
                            four_codes<FMT>(v[p].get(0) * s, v[p].get(1) * s, v[p].get(2) * s,
                                            v[p].get(3) * s),
                            four_codes<FMT>(v[p].get(4) * s, v[p].get(5) * s, v[p].get(6) * s,
                                            v[p].get(7) * s),
                            n, wide);
        }
    }
    if constexpr (WHAT & (kWriteCols | kWriteTiles)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t m = 0;
#pragma unroll
            for (int p = 0; p < 8; ++p) m = umax(m, finite_mag(v[p].get(e)));
            m = lane_max(m, 16, 64);
            if ((tid & 48) == 0) part[wave][c + e] = m;
        }
    }
    __syncthreads();
    if constexpr (WHAT & (kWriteCols | kWriteTiles)) {
        const bool wide = (lo32(cm.codes) & 7u) == 0 && (cm.ld & 7) == 0;
        float s[8];
        uint32_t all = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t m = umax(umax(part[0][c + e], part[1][c + e]),
                                    umax(part[2][c + e], part[3][c + e]));
            const uint32_t b = scale_byte<FMT>(m);
            all = umax(all, m);
            s[e] = inverse_scale(b);
            if constexpr (WHAT & kWriteCols)
                if (r == 0) bytes[1][c + e] = static_cast<uint8_t>(b);
        }
        if constexpr (WHAT & kWriteTiles) {
            const uint32_t b = scale_byte<FMT>(lane_max(all, 1, 16));
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = inverse_scale(b);
            if (tid == 0)
                cm.scales[static_cast<int64_t>(blockIdx.y) * cm.pitch + blockIdx.x] =
                    static_cast<uint8_t>(b);
        }
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const int row = r + 16 * p;
            if (row < rows)
                store_eight(cm.codes + static_cast<int64_t>(row0 + row) * cm.ld + col0 + c,
                            four_codes<FMT>(v[p].get(0) * s[0], v[p].get(1) * s[1],
                                            v[p].get(2) * s[2], v[p].get(3) * s[3]),
                            four_codes<FMT>(v[p].get(4) * s[4], v[p].get(5) * s[5],
                                            v[p].get(6) * s[6], v[p].get(7) * s[7]),
                            n, wide);
        }
        if constexpr (WHAT & kWriteCols) __syncthreads();
    }
    // The blocks' scales: neighbouring rows, or columns, are neighbouring bytes.
    if constexpr (WHAT & kWriteRows) {
        uint8_t *to = rm.scales + static_cast<int64_t>(blockIdx.x) * rm.pitch + row0;
        if (tid < 32 && 4 * tid + 4 <= rows)
            *reinterpret_cast<uint32_t *>(to + 4 * tid) =
                *reinterpret_cast<const uint32_t *>(&bytes[0][4 * tid]);
        else if (tid < 32)
            for (int k = 4 * tid; k < rows && k < 4 * tid + 4; ++k) to[k] = bytes[0][k];
    }
    if constexpr (WHAT & kWriteCols) {
        uint8_t *to = cm.scales + static_cast<int64_t>(blockIdx.y) * cm.pitch + col0;
        const int t = tid - 64;
        if (t >= 0 && t < 32 && 4 * t + 4 <= cols)
            *reinterpret_cast<uint32_t *>(to + 4 * t) =
                *reinterpret_cast<const uint32_t *>(&bytes[1][4 * t]);
        else if (t >= 0 && t < 32)
            for (int k = 4 * t; k < cols && k < 4 * t + 4; ++k) to[k] = bytes[1][k];
    }
}

// ---------------------------------------------------------------------------
// dequantise
// ---------------------------------------------------------------------------

template <int FMT>
__device__ __forceinline__ void code_values(uint32_t lo, uint32_t hi, float (&x)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int w = static_cast<int>(h ? hi : lo);
        if constexpr (FMT == FSDP_Q8_E4M3) {
            x[4 * h] = __builtin_amdgcn_cvt_f32_fp8(w, 0);
            x[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8(w, 1);
            x[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8(w, 2);
            x[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8(w, 3);
        } else {
            x[4 * h] = __builtin_amdgcn_cvt_f32_bf8(w, 0);
            x[4 * h + 1] = __builtin_amdgcn_cvt_f32_bf8(w, 1);
            x[4 * h + 2] = __builtin_amdgcn_cvt_f32_bf8(w, 2);
            x[4 * h + 3] = __builtin_amdgcn_cvt_f32_bf8(w, 3);
        }
    }
}

// The same blocks and threads.  A code times its power of two is exact in
// fp32; a divisor, where there is one, rounds once more.
template <int FMT, bool kF32>
__global__ __launch_bounds__(kBlock) void q8_dequantize_kernel(Q8Mat Q, void *__restrict__ out,
                                                               int64_t ldo) {
    const int tid = threadIdx.x, r = tid >> 4, c = (tid & 15) * 8;
    const int row0 = blockIdx.y * 128, col0 = blockIdx.x * 128;
    const int rows = Q.rows - row0 < 128 ? Q.rows - row0 : 128;
    const int cols = Q.cols - col0 < 128 ? Q.cols - col0 : 128;
    const int n = cols - c < 0 ? 0 : (cols - c < 8 ? cols - c : 8);
    if (n == 0) return;
    const bool vec = n == 8 && (lo32(Q.codes) & 7u) == 0 && (Q.ld & 7) == 0;
    const bool wide = n == 8 && (lo32(out) & 15u) == 0 && (ldo & (kF32 ? 3 : 7)) == 0;
    const float div = Q.divisor ? *Q.divisor : 1.0f;
    float s[8];
    const uint8_t *sb = Q.scales + (Q.blocks == FSDP_Q8_ROWS
                                        ? static_cast<int64_t>(blockIdx.x) * Q.pitch
                                        : static_cast<int64_t>(blockIdx.y) * Q.pitch);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        s[e] = Q.blocks == FSDP_Q8_COLS    ? scale_of(sb[col0 + c + (e < n ? e : 0)])
               : Q.blocks == FSDP_Q8_TILES ? scale_of(sb[blockIdx.x])
                                           : 1.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int row = r + 16 * p;
        if (row >= rows) continue;
        const uint8_t *from = Q.codes + static_cast<int64_t>(row0 + row) * Q.ld + col0 + c;
        uint32_t w[2] = {0u, 0u};
        if (vec) {
            const u32x2 t = *reinterpret_cast<const u32x2 *>(from);
            w[0] = t.x;
            w[1] = t.y;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) w[e >> 2] |= static_cast<uint32_t>(from[e]) << (8 * (e & 3));
        }
        const float sr = Q.blocks == FSDP_Q8_ROWS ? scale_of(sb[row0 + row]) : 1.0f;
        float y[8];
        code_values<FMT>(w[0], w[1], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[e] *= Q.blocks == FSDP_Q8_ROWS ? sr : s[e];
            if (Q.divisor) y[e] /= div;
        }
        const int64_t o = static_cast<int64_t>(row0 + row) * ldo + col0 + c;
        if constexpr (kF32) {
            float *to = static_cast<float *>(out) + o;
            if (wide) {
                reinterpret_cast<f32x4 *>(to)[0] = f32x4{y[0], y[1], y[2], y[3]};
                reinterpret_cast<f32x4 *>(to)[1] = f32x4{y[4], y[5], y[6], y[7]};
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) to[e] = y[e];
            }
        } else {
            uint16_t *to = static_cast<uint16_t *>(out) + o;
            const u32x4 h = pack8(y);
            if (wide) {
                *reinterpret_cast<u32x4 *>(to) = h;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) to[e] = static_cast<uint16_t>(h[e >> 1] >> (16 * (e & 1)));
            }
        }
    }
}

// ---------------------------------------------------------------------------
// FP8 copy-in with block scales
// ---------------------------------------------------------------------------

// One block's part on this rank a workgroup: 32 lanes take a row's 128 columns,
// four each.  Cells of entry -1 are blocks that other ranks hold alone: zeros.
__global__ __launch_bounds__(kBlock) void block_scales_kernel(
    const BlockCell *__restrict__ cells, int64_t n_cells, const BlockEntry *__restrict__ blocks,
    const DevEntry *__restrict__ ents, uint8_t *__restrict__ scales) {
  __shared__ uint32_t part[4];
  for (int64_t k = blockIdx.x; k < n_cells; k += gridDim.x) {
    const BlockCell cell = cells[k];
    const int tid = threadIdx.x;
    if (cell.entry < 0) {
        for (int i = tid; i < cell.rows; i += kBlock) scales[cell.at + i] = 0;
        continue;
    }
    const int64_t width = blocks[cell.entry].cols;
    const float *p = ents[cell.entry].master + cell.row * width + cell.col;
    const int64_t left = width - cell.col;
    const int c = (tid & 31) * 4, n = left - c < 0 ? 0 : (left - c < 4 ? static_cast<int>(left - c) : 4);
    const bool vec = n == 4 && (lo32(p) & 15u) == 0 && (width & 3) == 0;
    uint32_t m = 0;
    if (vec) {
#pragma unroll 4
        for (int r = tid >> 5; r < cell.rows; r += 8) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(p + r * width + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) m = umax(m, finite_mag(v[e]));
        }
    } else {
        for (int r = tid >> 5; r < cell.rows; r += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n) m = umax(m, finite_mag(p[r * width + c + e]));
    }
    m = lane_max(m, 1, 64);
    __syncthreads();            // the cell before is done with `part`
    if ((tid & 63) == 0) part[tid >> 6] = m;
    __syncthreads();
    if (tid == 0)
        scales[cell.at] = static_cast<uint8_t>(
            scale_byte<FSDP_Q8_E4M3>(umax(umax(part[0], part[1]), umax(part[2], part[3]))));
  }
}

// Row and column that lie d elements after column `col` of row `row`.
struct Place {
    int64_t row, col;
};
__device__ __forceinline__ Place place_after(int64_t row, int64_t col, uint32_t d, int64_t cols) {
    const int64_t x = col + d;
    if (x < cols) return {row, x};
    // here cols <= col + d; a tile is at most 2^14 long
    if (cols > (1 << 20)) return {row + 1, x - cols};
    const uint32_t q = static_cast<uint32_t>(x) / static_cast<uint32_t>(cols);
    return {row + q, x - static_cast<int64_t>(q) * cols};
}

// Sixteen codes a lane.  Where a lane's sixteen lie in one block it reads one
// scale, otherwise one for each element.
__global__ __launch_bounds__(kBlock) void pack_fp8_blocks_kernel(
    const PackTile *__restrict__ tiles, int64_t n_tiles, int32_t split, int64_t sub,
    const BlockEntry *__restrict__ blocks, const DevEntry *__restrict__ ents,
    uint8_t *__restrict__ ag_in, const uint8_t *__restrict__ scales) {
    const int64_t nvt = n_tiles * split;
    for (int64_t vt = first_vt(); vt < nvt; vt += gridDim.x) {
        int64_t t, b;
        sub_range(vt, split, sub, &t, &b);
        const PackTile tl = tiles[t];
        if (b >= tl.len) continue;
        const int len = static_cast<int>(tl.len - b < sub ? tl.len - b : sub);
        const int64_t left = tl.valid - b;
        const int valid = left < 0 ? 0 : (left > len ? len : static_cast<int>(left));
        const BlockEntry be = blocks[tl.entry];
        const int64_t first = tl.src + b;
        const int64_t row0 = first / be.cols, col0 = first - row0 * be.cols;
        const int64_t across = (be.cols + 127) >> 7;
        const float *src = ents[tl.entry].master + first;
        uint8_t *dst = ag_in + tl.dst + b;
        auto scale_at = [&](const Place &at) {
            return inverse_scale(
                scales[be.at + ((be.row_begin + at.row) >> 7) * across + (at.col >> 7)]);
        };
        // bytes before the first 16-byte boundary of the destination, and the last ones
        int head = static_cast<int>((16u - (lo32(dst) & 15u)) & 15u);
        head = head < valid ? head : valid;
        const int groups = (valid - head) >> 4, done = head + groups * 16;
        auto one = [&](int i) {
            const float v = src[i] * scale_at(place_after(row0, col0, i, be.cols));
            dst[i] = static_cast<uint8_t>(four_codes<FSDP_Q8_E4M3>(v, v, v, v));
        };
        const int tid = threadIdx.x;
        if (tid < head) one(tid);
        if (tid < valid - done) one(done + tid);
        const uint32_t q = (lo32(src + head) >> 2) & 3u;
        for (int g = tid; g < groups; g += kBlock) {
            const int o = head + g * 16;
            f32x4 v[4];
            if (q == 0) {
                load8f<0, true>(src + o, 0u, v[0], v[1]);
                load8f<0, true>(src + o + 8, 0u, v[2], v[3]);
            } else {
                load8f<0, false>(src + o, q, v[0], v[1]);
                load8f<0, false>(src + o + 8, q, v[2], v[3]);
            }
            Place at = place_after(row0, col0, o, be.cols);
            u32x4 w;
            if (at.col + 16 <= be.cols && (at.col & 127) <= 112) {
                const float s = scale_at(at);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = four_codes<FSDP_Q8_E4M3>(v[k].x * s, v[k].y * s, v[k].z * s, v[k].w * s);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[e] = v[k][e] * scale_at(at);
                        if (++at.col == be.cols) at = {at.row + 1, 0};
                    }
                    w[k] = four_codes<FSDP_Q8_E4M3>(y[0], y[1], y[2], y[3]);
                }
            }
            *reinterpret_cast<u32x4 *>(dst + o) = w;
        }
        for (int i = valid + tid; i < len; i += kBlock) dst[i] = 0;
    }
}

template <int FMT, bool kF32>
void quantize(const void *x, int64_t ldx, const Q8Mat &a, const Q8Mat *b, dim3 grid,
              hipStream_t st) {
    const Q8Mat none{};
    const Q8Mat &second = b ? *b : none;
    if (b != nullptr)
        q8_quantize_kernel<FMT, kF32, kWriteRows | kWriteCols>
            <<<grid, kBlock, 0, st>>>(x, ldx, a, second);
    else if (a.blocks == FSDP_Q8_ROWS)
        q8_quantize_kernel<FMT, kF32, kWriteRows><<<grid, kBlock, 0, st>>>(x, ldx, a, second);
    else if (a.blocks == FSDP_Q8_COLS)
        q8_quantize_kernel<FMT, kF32, kWriteCols><<<grid, kBlock, 0, st>>>(x, ldx, a, second);
    else
        q8_quantize_kernel<FMT, kF32, kWriteTiles><<<grid, kBlock, 0, st>>>(x, ldx, a, second);
}

dim3 blocks_of(const Q8Mat &m) { return dim3((m.cols + 127) / 128, (m.rows + 127) / 128); }

}  // namespace

hipError_t launch_q8_quantize(const void *x, bool f32, int64_t ldx, const Q8Mat &a, const Q8Mat *b,
                              hipStream_t st) {
    if (a.rows == 0 || a.cols == 0) return hipSuccess;
    const Q8Mat &rows = b && a.blocks == FSDP_Q8_COLS ? *b : a;
    const Q8Mat *cols = b && a.blocks == FSDP_Q8_COLS ? &a : b;
    const dim3 grid = blocks_of(a);
    if (a.format == FSDP_Q8_E4M3)
        f32 ? quantize<FSDP_Q8_E4M3, true>(x, ldx, rows, cols, grid, st)
            : quantize<FSDP_Q8_E4M3, false>(x, ldx, rows, cols, grid, st);
    else
        f32 ? quantize<FSDP_Q8_E5M2, true>(x, ldx, rows, cols, grid, st)
            : quantize<FSDP_Q8_E5M2, false>(x, ldx, rows, cols, grid, st);
    return hipGetLastError();
}

hipError_t launch_q8_dequantize(const Q8Mat &q, void *out, bool f32, int64_t ldo, hipStream_t st) {
    if (q.rows == 0 || q.cols == 0) return hipSuccess;
    const dim3 grid = blocks_of(q);
    if (q.format == FSDP_Q8_E4M3)
        f32 ? q8_dequantize_kernel<FSDP_Q8_E4M3, true><<<grid, kBlock, 0, st>>>(q, out, ldo)
            : q8_dequantize_kernel<FSDP_Q8_E4M3, false><<<grid, kBlock, 0, st>>>(q, out, ldo);
    else
        f32 ? q8_dequantize_kernel<FSDP_Q8_E5M2, true><<<grid, kBlock, 0, st>>>(q, out, ldo)
            : q8_dequantize_kernel<FSDP_Q8_E5M2, false><<<grid, kBlock, 0, st>>>(q, out, ldo);
    return hipGetLastError();
}

hipError_t launch_block_scales(const BlockCell *cells, int64_t n, const BlockEntry *blocks,
                               const DevEntry *ents, uint8_t *scales, hipStream_t st) {
    if (n == 0) return hipSuccess;
    block_scales_kernel<<<grid_for(n, 1), kBlock, 0, st>>>(cells, n, blocks, ents, scales);
    return hipGetLastError();
}

hipError_t launch_pack_fp8_blocks(const PackTile *tiles, int64_t n, const BlockEntry *blocks,
                                  const DevEntry *ents, uint8_t *ag_in, const uint8_t *scales,
                                  hipStream_t st) {
    if (n == 0) return hipSuccess;
    const int32_t sp = split_for(kTilePack, 4096);
    pack_fp8_blocks_kernel<<<grid_for(n, sp), kBlock, 0, st>>>(tiles, n, sp, kTilePack / sp, blocks,
                                                               ents, ag_in, scales);
    return hipGetLastError();
}

}  // namespace fsdp
