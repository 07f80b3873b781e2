// Orthogonalisation of matrices by Newton-Schulz products, on the matrix
// cores.  For X = U/(|U|_F + eps), m x n with m <= n (a tall U is worked on
// transposed), each iteration is
//
//   A = X X^T        m x m, symmetric: the lower triangle of tiles
//   B = b A + c A A  m x m, symmetric as well
//   X = a X + B X    m x n
//
// Precision.  Products take fp16 operands and add in fp32: 11 bits against
// bf16's 8 at the same rate, with the matrices scaled by powers of two into
// fp16's range (X by 2^12 and more, A and B by 2^11).  A direction whose
// singular value is still small is multiplied by a in every iteration, 3.4445^5
// = 485 times in all, and so is whatever rounding X adds to it: with X held in
// fp16 alone the result was 3.5e-3 off for a falling spectrum and 2.7e-2 for
// one of low rank (relative, in the Frobenius norm; bf16 1e-2 to 0.2).  The term a X
// therefore takes X as a high and a low fp16 part (22 bits); the products,
// which vanish with the singular value, take the high part.  That leaves 3e-4
// to 2e-3 on gradients, noise and falling spectra, where the roundings of X, A
// and B are independent of each other: below the 1.7e-3 of rounding the result
// to bf16 itself or near it.  Where many entries have the same magnitude their
// roundings are the same, and add up: 2e-3 to 8e-3 on constants, signs of rank
// one, repeated or orthonormal rows and identities, 1.7e-2 on two constants in
// blocks.
//
// A plan may therefore have its products made of both parts of every operand,
// in three terms (high high, low high, high low), like those of few rows below:
// 22 bits throughout, 1e-6 to 3e-5 off on all of these, in 2.3 to 2.9 times the
// time (a decoder block's seven matrices 39.1 ms for 14.7).
//
// Layout.  Only X^T is stored.  X = a X + B X is then a product of rows with
// rows (rows of B, rows of X^T), and A sums over rows of X^T, whose tiles the
// transposing LDS read turns into operands.  X^T, A and B lie in panels of 32
// columns, [columns / 32][rows][32]: the rows of one step of a sum (64 bytes
// each) follow each other, and so do a 32 x 32 block's in an epilogue.
#include "ortho.hpp"

#include "device.hpp"

namespace fsdp {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) s16x8 lds_s16x8;
typedef __attribute__((address_space(3))) f16x4 lds_f16x4;
typedef __attribute__((address_space(3))) f16x8 lds_f16x8;

// log2 of the scale of A and B
constexpr int kLogA = 11;
// log2 of the scale of X where the norm is not lost in eps
constexpr int kLogX = 12;

__device__ __forceinline__ char *at(void *ws, int64_t off) { return static_cast<char *>(ws) + off; }

// x as one fp32 value.  Without this the compiler may take a product and its
// conversion to fp16 as one operation of one rounding in one place and as two
// in another, and a high part that is stored then differs, where the two
// round apart, from the one that the low part was taken against.
__device__ __forceinline__ float settled(float x) {
    asm volatile("" : "+v"(x));
    return x;
}

// To nearest even, by the instruction: no branch for NaN.
__device__ __forceinline__ uint16_t to_bf16(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}

// Element (row, col) of a matrix in panels of 32 columns with `rows` rows.
__device__ __forceinline__ int64_t panel_at(int rows, int row, int col) {
    return (static_cast<int64_t>(col >> 5) * rows + row) * 32 + (col & 31);
}

// ---------------------------------------------------------------------------
// norm and start
// ---------------------------------------------------------------------------

template <bool kF32>
__device__ __forceinline__ float load_in(const void *in, int64_t i) {
    if constexpr (kF32) return static_cast<const float *>(in)[i];
    else return widen(static_cast<const uint16_t *>(in)[i]);
}

// Sum over the block in a fixed order; every thread gets it.
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double part[kBlock / 64];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kBlock / 64; ++w) s += part[w];
    return s;
}

// Eight neighbouring values from i; one load, or two, where `vec` says that
// they may be.
template <bool kF32>
__device__ __forceinline__ void load_in8(const void *in, int64_t i, bool vec, float (&x)[8]) {
    if constexpr (kF32) {
        const float *p = static_cast<const float *>(in) + i;
        if (vec) {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(p);
            const f32x4 b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = a[e], x[e + 4] = b[e];
            return;
        }
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(in) + i;
        if (vec) {
            const u32x4 w = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[2 * e] = bf16_lo(w[e]), x[2 * e + 1] = bf16_hi(w[e]);
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = load_in<kF32>(in, i + e);
}

// Sums of squares in fp64: no scaling is needed for the smallest and largest
// values, and the order is fixed.  Parts start at multiples of eight elements,
// and a thread has four loads of eight under way.
template <bool kF32>
__global__ __launch_bounds__(kBlock) void ortho_norm_kernel(const OrthoTile *__restrict__ tiles,
                                                            const OrthoMat *__restrict__ mats,
                                                            void *ws) {
    const OrthoTile tl = tiles[blockIdx.x];
    const OrthoMat M = mats[tl.mat];
    const int64_t total = static_cast<int64_t>(M.rows) * M.cols, eights = total >> 3;
    const int64_t per = (eights + M.n_parts - 1) / M.n_parts;
    const int64_t lo = per * tl.ti, hi = lo + per < eights ? lo + per : eights;
    const bool vec = (lo32(M.in) & 15u) == 0;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    for (int64_t i = lo + threadIdx.x; i < hi; i += 4 * kBlock) {
        // past the end the first eight again, which count nothing: no branch lies
        // between the loads
        float x[4][8];
#pragma unroll
        for (int t = 0; t < 4; ++t)
            load_in8<kF32>(M.in, (i + t * kBlock < hi ? i + t * kBlock : lo) * 8, vec, x[t]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const bool in = i + t * kBlock < hi;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double d = in ? x[t][e] : 0.0f;
                s[t] = __builtin_fma(d, d, s[t]);       // the product is exact
            }
        }
    }
    if (tl.ti == M.n_parts - 1 && eights * 8 + threadIdx.x < total) {
        const double x = load_in<kF32>(M.in, eights * 8 + threadIdx.x);
        s[0] += x * x;
    }
    const double sum = block_sum((s[0] + s[1]) + (s[2] + s[3]));
    if (threadIdx.x == 0) reinterpret_cast<double *>(at(ws, M.parts))[tl.ti] = sum;
}

// The scalars of a matrix from its norm: X = U / (norm + eps) is stored as U
// 2^k, which puts the norm at 2^kLogX or up to twice that.  X is small where
// eps outweighs the norm; up to what the iterations can magnify it back
// (2^growth), it is scaled up instead.  A norm that is not finite makes the
// scalars NaN and so every output; the stored X is then to be zero.
__device__ __forceinline__ OrthoScal scalars(double norm, double eps, int32_t growth, int *k) {
    OrthoScal s{__builtin_nanf(""), 0.0f, __builtin_nanf(""), 0.0f};
    *k = 0;
    if (!isfinite(norm)) return s;
    int e = 0, up = 0;
    double p0 = eps > 0.0 ? 1.0 : s.phi0;       // X = stored * p0; zero / 0 is NaN
    if (norm > 0.0) {
        e = ilogb(norm);
        const double r = norm / (norm + eps);
        up = r > 0.0 ? -ilogb(r) - growth : 100;
        up = up < 0 ? 0 : (up > 100 ? 100 : up);
        p0 = 1.0 / ldexp(norm + eps, kLogX - e);
    }
    *k = kLogX - e;
    s.phi = ldexpf(1.0f, -(kLogX + up));
    s.phi0 = static_cast<float>(p0);
    s.rho = static_cast<float>(ldexp(p0, kLogX + up));
    return s;
}

// Four rows of 16 columns: lane l of a 16-lane group reads 4 neighbouring
// columns (8 bytes at t) of row l >> 2, and gets column l of the 16 that lanes
// 0 to 3 read, of those 4 rows.  (restrict: with aliasing facts on the read the
// compiler does not wait for every load to LDS that is under way before it;
// the borders wait for those that matter.)
__device__ __forceinline__ s16x4 read_tr(lds_char *__restrict__ t) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)t);
}

// X^T's 64 x 64 pieces tj .. + part of n for piece ti of m, one after the other, the
// next one's values under way: the norm's parts are summed once for all of them.
// Eight neighbouring values a thread and turn: of a tall U as they lie, of a wide one
// turned over by transposing LDS reads.  A bf16 input times 2^k is an fp16 value but
// for what lies under 2^-26 of the norm (2^-37 of the norm at most is lost there);
// an fp32 input leaves a low part.
template <bool kF32>
__global__ __launch_bounds__(kBlock) void ortho_init_kernel(const OrthoTile *__restrict__ tiles,
                                                            const OrthoMat *__restrict__ mats,
                                                            void *ws, double eps, int32_t growth) {
    constexpr int kParts = kF32 ? 2 : 1, kPitch = 72;
    // two pieces in turn: one barrier a piece
    __shared__ __attribute__((aligned(16))) _Float16 buf[2][kParts][64 * kPitch];
    const OrthoTile tl = tiles[blockIdx.x];
    const OrthoMat M = mats[tl.mat];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool vec = (lo32(M.in) & 15u) == 0 && (M.cols & 7) == 0;
    float x[2][8];
    auto load = [&](int piece) {
        const int r0 = (M.wide ? tl.ti : piece) * 64, c0 = (M.wide ? piece : tl.ti) * 64;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int u = t * kBlock + threadIdx.x, r = r0 + (u >> 3), c = c0 + (u & 7) * 8;
            const int64_t o = static_cast<int64_t>(r) * M.cols + c;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[t][e] = 0.0f;
            if (r < M.rows && c + 8 <= M.cols) {
                load_in8<kF32>(M.in, o, vec, x[t]);
            } else if (r < M.rows) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < M.cols) x[t][e] = load_in<kF32>(M.in, o + e);
            }
        }
    };
    load(tl.tj);
    const double *parts = reinterpret_cast<const double *>(at(ws, M.parts));
    double s = 0.0;
    for (int i = threadIdx.x; i < M.n_parts; i += kBlock) s += parts[i];
    const double norm = sqrt(block_sum(s));
    const bool fine = isfinite(norm);
    int k;
    const OrthoScal sc = scalars(norm, eps, growth, &k);
    if (tl.ti == 0 && tl.tj == 0 && threadIdx.x == 0)
        *reinterpret_cast<OrthoScal *>(at(ws, M.scal)) = sc;
    f16x8 *hi = reinterpret_cast<f16x8 *>(at(ws, M.t[0]));
    f16x8 *lo = reinterpret_cast<f16x8 *>(at(ws, M.lo));
    for (int piece = tl.tj; piece < tl.tj + tl.part; ++piece) {
        f16x8 h[2], l[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = fine ? settled(ldexpf(x[t][e], k)) : 0.0f;
                h[t][e] = static_cast<_Float16>(f);
                l[t][e] = static_cast<_Float16>(f - static_cast<float>(h[t][e]));
            }
        if (piece + 1 < tl.tj + tl.part) load(piece + 1);
        if (!M.wide) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int u = t * kBlock + threadIdx.x, y = u >> 3, c = (u & 7) * 8;
                const int64_t o = panel_at(M.np, piece * 64 + y, tl.ti * 64 + c) >> 3;
                hi[o] = h[t];
                if constexpr (kF32) lo[o] = l[t];
            }
            continue;
        }
        _Float16(&now)[kParts][64 * kPitch] = buf[piece & 1];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int u = t * kBlock + threadIdx.x, o = (u >> 3) * kPitch + (u & 7) * 8;
            *reinterpret_cast<f16x8 *>(&now[0][o]) = h[t];
            if constexpr (kF32) *reinterpret_cast<f16x8 *>(&now[kParts - 1][o]) = l[t];
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            // 16 rows y of X^T, 32 of its columns: 1 KB that a wave writes whole
            const int y = wave * 16, c = t * 32 + (lane >> 4) * 8;
            const int from = (c + ((lane >> 2) & 3)) * kPitch + y + (lane & 3) * 4;
            const int64_t o = panel_at(M.np, piece * 64 + y + (lane & 15), tl.ti * 64 + c) >> 3;
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                lds_char *b = (lds_char *)&now[part][from];
                union {
                    s16x4 q[2];
                    f16x8 f;
                } v;
                v.q[0] = read_tr(b);
                v.q[1] = read_tr(b + 4 * kPitch * 2);
                (part == 0 ? hi : lo)[o] = v.f;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

// when: the first iteration; X has no low part yet (bf16 inputs)
enum { kFirst = 1, kHigh = 2 };
// kGramPart: a stretch of kGram's sum, left in fp32; kGramJoin: their sum
enum { kGram = 0, kPoly = 1, kApply = 2, kLast = 3, kGramPart = 4, kGramJoin = 5 };

// elements of the sum per stage: one panel of columns
constexpr int kBK = 32;

// Blocks of 32 x 32 are two by two products of 16 x 16 (and 32 of the sum).  Of
// a product's 16 rows lane l gets back 4 (l >> 4) .. + 4, so the rows of half b
// of a block are taken in an order that joins the two halves' fours to eight
// neighbouring rows: 16-byte stores.
__device__ __forceinline__ int perm_row(int r, int b) { return 8 * (r >> 2) + 4 * b + (r & 3); }

// Rows of 64 bytes in LDS: a row's 16-byte chunk sits at its index xor this.  One
// LDS cycle serves 16 lanes of which half come from the other 16 of each 32
// (measured by conflicts: quads 0, 2 with 5, 7 and so on), which read the next
// chunk: with the two 16-row halves apart they hit all 64 banks.
__device__ __forceinline__ int swz_row(int row) { return ((row >> 4) & 1) << 1; }

// Rows of a panel into LDS, straight from memory: load u of a tile writes 1 KB,
// the rows 16 u .. 16 u + 16.  Past nbytes it writes zeros.
__device__ __forceinline__ void fill_rows(lds_char *dst, const char *src, uint32_t nbytes, int u,
                                          int lane) {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(src), 0, nbytes, 0x00020000);
    const uint32_t voff = static_cast<uint32_t>(
        (lane >> 2) * 64 + ((lane & 3) ^ swz_row(16 * (u & 1) + (lane >> 2))) * 16);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(dst + u * 1024), 16, voff, u * 1024, 0,
                                             0);
}

// Where the sum runs over rows: the halves of a row's 64 bytes change places in
// every other eight rows, so that the 32 lanes of one LDS cycle, which read 32
// bytes each of four rows and of four rows eight further, hit all banks.
__device__ __forceinline__ int swz_col(int k) { return (k >> 3) & 1; }

// The rows [32 s, 32 s + 32) of panels of `panel` bytes each, in LDS one
// panel's 2 KB after the other; load u: half a panel's.
__device__ __forceinline__ void fill_cols(lds_char *dst, const char *src, uint32_t nbytes,
                                          uint32_t panel, int s, int u, int lane) {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(src), 0, nbytes, 0x00020000);
    const uint32_t voff = static_cast<uint32_t>((lane ^ (swz_col(lane >> 2) << 1)) * 16);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, (lds_void *)(dst + u * 1024), 16, voff,
        static_cast<uint32_t>(u >> 1) * panel + (u & 1) * 1024 + s * 2048, 0, 0);
}

// Operand of 16 rows and 32 elements of the sum: this lane's row, its 8.
__device__ __forceinline__ f16x8 read_rows(const lds_char *t, int row, int lane) {
    return *(const lds_f16x8 *)(t + row * 64 + ((lane >> 4) ^ swz_row(row)) * 16);
}

// The operand from a tile with the sum over rows, of 16 neighbouring columns
// from col.
__device__ __forceinline__ f16x8 read_cols(lds_char *t, int col, int lane) {
    const int k = (lane >> 4) * 8 + ((lane >> 2) & 3);
    lds_char *at = t + (col >> 5) * 2048 + k * 64 +
                   ((((col >> 4) & 1) ^ swz_col(k)) * 32) + (lane & 3) * 8;
    union {
        s16x4 s[2];
        f16x8 v;
    } u;
    u.s[0] = read_tr(at);
    u.s[1] = read_tr(at + 4 * 64);
    return u.v;
}

union Half8 {
    f16x8 f;
    s16x8 s;
    s16x4 q[2];
    u32x4 w;
};

// n of 8 bf16 at p, in one store where they are all there and p allows it.
__device__ __forceinline__ void store_out(uint16_t *p, const Half8 &v, int n, bool vec) {
    if (vec && n >= 8) {
        *reinterpret_cast<u32x4 *>(p) = v.w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = static_cast<uint16_t>(v.s[e]);
    }
}

template <int N>
struct Int {
    static constexpr int value = N;
};

template <int N>
__device__ __forceinline__ void border() {
    // vmcnt(N) lgkmcnt(0), then the barrier
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// C = alpha * (sums of P's rows i with Q's rows j), one BM x BN tile a block.
//
// NST stages of LDS, of which NST - 1 are on their way while one is read.  A
// stage's products are made in two parts, for the first and the second half of
// the wave's rows i; while the matrix cores work on one part the operands of
// the next are read, across the stages' borders too (rows j alternate between
// two sets of registers).  At a border every wave has its last operands of the
// old stage in registers (lgkmcnt) and its loads of the next one landed
// (vmcnt: those after it may be under way); past the barrier the next stage
// may be read and the old one overwritten.
//
// kFine: operands as high and low parts.  The sum is three times as long, over
// (high, high), (low, high) and (high, low) parts one after the other: the terms
// differ only in the memory that a stage is filled from.
template <int KIND, int BM, int BN, int WM, int WN, bool kFine>
__global__ __launch_bounds__(64 * WM *WN) void ortho_product_kernel(
    const OrthoTile *__restrict__ tiles, const OrthoMat *__restrict__ mats, void *ws, int32_t src,
    int32_t when, int32_t split, OrthoCoef coef) {
    constexpr int WAVES = WM * WN, WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
    constexpr int NST = 4;
    constexpr bool kXXT = KIND == kGram || KIND == kGramPart || KIND == kGramJoin;
    constexpr bool kSym = kXXT || KIND == kPoly;
    constexpr int kStage = (BM + BN) * kBK * 2, kLoadsP = BM / 16 / WAVES,
                  kLoadsQ = BN / 16 / WAVES;
    static_assert(BM % (16 * WAVES) == 0 && BN % (16 * WAVES) == 0, "whole loads per wave");
    static_assert(NST * kStage >= WAVES * 2048 && kBK == 32 && FM % 2 == 0 && FN % 2 == 0, "");
    __shared__ __attribute__((aligned(1024))) char smem[NST * kStage];
    lds_char *lds = (lds_char *)smem;

    const OrthoTile tl = tiles[blockIdx.x];
    const OrthoMat M = mats[tl.mat];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int i0 = tl.ti * BM, j0 = tl.tj * BN;
    const int g = lane >> 4;
    const OrthoScal sc = *reinterpret_cast<const OrthoScal *>(at(ws, M.scal));
    const char *T = at(ws, src ? M.t[1] : M.t[0]);
    // X's low part: in place where nothing but a X reads it
    const char *L = at(ws, kFine && src ? M.lo2 : M.lo);

    f32x4 acc[FM][FN];
    if constexpr (KIND == kGramJoin) {
        // the parts in order
        const f32x4 *part = reinterpret_cast<const f32x4 *>(at(ws, M.sums)) +
                            static_cast<int64_t>(tl.part) * (BM * BN / 4) + threadIdx.x;
#pragma unroll
        for (int x = 0; x < FM; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y) acc[x][y] = part[(x * FN + y) * 64 * WAVES];
        for (int k = 1; k < split; ++k) {
            part += BM * BN / 4;
#pragma unroll
            for (int x = 0; x < FM; ++x)
#pragma unroll
                for (int y = 0; y < FN; ++y) acc[x][y] += part[(x * FN + y) * 64 * WAVES];
        }
    } else {
        // stages of the sum, or of this part's stretch of it, a multiple of four: of
        // one term, and of all
        int term = (kXXT ? M.np : M.mp) / kBK, steps;
        const char *TH = T, *TL = L;
        if constexpr (KIND == kGramPart) {
            const int units = term / NST, k = tl.part % split;
            const int from = units * k / split, to = units * (k + 1) / split;
            TH += static_cast<int64_t>(from) * NST * 2048;
            TL += static_cast<int64_t>(from) * NST * 2048;
            term = (to - from) * NST;
        }
        steps = term;
        if constexpr (kFine) {
            // before the first iteration a bf16 input has no low part
            const bool high = KIND != kPoly && (when & kFirst) && !M.low;
            steps = term * (!high ? 3 : kXXT ? 1 : 2);
        }
        // The part of an operand that stage s is filled from, and its stage within the
        // term; second: the low part's turn.
        auto source = [&](const char *high, const char *low, int second, int &s) {
            if constexpr (kFine) {
                const int t = (s >= term) + (s >= 2 * term);
                s -= t * term;
                return t == second ? low : high;
            } else {
                return high;
            }
        };
        // load k of this wave's kLoadsP of stage s's rows i, or of its kLoadsQ of the rows j
        auto fill_p = [&](int s, int k) {
            lds_char *b = lds + (s & (NST - 1)) * kStage;
            const int u = k * WAVES + wave;
            if constexpr (kXXT) {
                // rows of X^T are the sum, columns i and j
                const uint32_t panel = static_cast<uint32_t>(M.np) * 64u;
                const int at = i0 / 32, n = M.mp / 32 - at < BM / 32 ? M.mp / 32 - at : BM / 32;
                const char *X = source(TH, TL, 1, s);
                fill_cols(b, X + static_cast<int64_t>(at) * panel, n * panel, panel, s, u, lane);
            } else {
                const char *A = source(at(ws, KIND == kPoly ? M.a : M.b),
                                       at(ws, KIND == kPoly ? M.al : M.bl), 1, s);
                const int n = M.mp - i0 < BM ? M.mp - i0 : BM;
                fill_rows(b, A + (static_cast<int64_t>(s) * M.mp + i0) * 64, n * 64u, u, lane);
            }
        };
        auto fill_q = [&](int s, int k) {
            lds_char *b = lds + (s & (NST - 1)) * kStage + BM * 64;
            const int u = k * WAVES + wave;
            if constexpr (kXXT) {
                const uint32_t panel = static_cast<uint32_t>(M.np) * 64u;
                const int at = j0 / 32, n = M.mp / 32 - at < BN / 32 ? M.mp / 32 - at : BN / 32;
                const char *X = source(TH, TL, 2, s);
                fill_cols(b, X + static_cast<int64_t>(at) * panel, n * panel, panel, s, u, lane);
            } else {
                const char *A = source(KIND == kPoly ? at(ws, M.a) : T,
                                       KIND == kPoly ? at(ws, M.al) : L, 2, s);
                const int rq = KIND == kPoly ? M.mp : M.np, n = rq - j0 < BN ? rq - j0 : BN;
                fill_rows(b, A + (static_cast<int64_t>(s) * rq + j0) * 64, n * 64u, u, lane);
            }
        };
        f16x8 p[2][FM / 2], q[2][FN];
        // operand k of part h of stage s's rows i; of its rows j, into set `set`
        auto read_p = [&](int s, int h, int k) {
            lds_char *t = lds + (s & (NST - 1)) * kStage;
            const int x = h * (FM / 2) + k, base = wm * WTM + (x >> 1) * 32;
            if constexpr (kXXT) p[h][k] = read_cols(t, base + (x & 1) * 16, lane);
            else p[h][k] = read_rows(t, base + perm_row(lane & 15, x & 1), lane);
        };
        auto read_q = [&](int s, int set, int y) {
            lds_char *t = lds + (s & (NST - 1)) * kStage + BM * 64;
            const int base = wn * WTN + (y >> 1) * 32;
            if constexpr (kXXT) q[set][y] = read_cols(t, base + (y & 1) * 16, lane);
            else q[set][y] = read_rows(t, base + perm_row(lane & 15, y & 1), lane);
        };

#pragma unroll
        for (int s = 0; s < NST - 1; ++s) {
#pragma unroll
            for (int k = 0; k < kLoadsP; ++k) fill_p(s, k);
#pragma unroll
            for (int k = 0; k < kLoadsQ; ++k) fill_q(s, k);
        }
        // Pair n of a X: two 16 x 16 blocks, rows 8 g .. + 8 of one column j a lane.
        auto load_x = [&](int n, f16x8 &hi, f16x8 &lo) {
            const int x = n / FN * 2, y = n % FN;
            // of one panel, through its range: past the matrix, and of a low part
            // that there is not, zeros
            const int at32 = (i0 + wm * WTM) / 32 + x / 2;
            const int j = j0 + wn * WTN + (y >> 1) * 32 + perm_row(lane & 15, y & 1);
            const int64_t panel = static_cast<int64_t>(at32) * M.np * 64;
            const uint32_t n32 = at32 < M.mp / 32 ? static_cast<uint32_t>(M.np) * 64u : 0u;
            const uint32_t o = static_cast<uint32_t>(j) * 64u + 16u * g;
            hi = __builtin_bit_cast(f16x8, bload16<0>(T + panel, o, n32));
            lo = __builtin_bit_cast(
                f16x8, bload16<0>(L + panel, o, when & kHigh ? 0u : n32));
        };
        auto add_x = [&](int n, const f16x8 &hi, const f16x8 &lo) {
            const float ca = ldexpf(coef.a, kLogA);
            const int x = n / FN * 2, y = n % FN;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                acc[x + (e >> 2)][y][e & 3] +=
                    ca * (static_cast<float>(hi[e]) + static_cast<float>(lo[e]));
        };
        // a X: where a CU has one block, whose loads of it nothing else covers, two pairs
        // at a time in eight turns along the sum (two 1024 x 8192: 511 -> 490 us, a
        // decoder block's 15.3 -> 15.1 ms); as the sums' start where blocks share a CU
        // or the sum is short.  A border's wait counts the loads younger than a stage's;
        // these between only make it longer.
        constexpr int kPairs = FM / 2 * FN, kTurns = kPairs / 2;
        constexpr bool kSpread = !kSym && BM == 256;
        const bool spread = kSpread && steps >= 4 + 2 * kTurns;
#pragma unroll
        for (int x = 0; x < FM; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (!kSym && !spread) {
#pragma unroll
            for (int n = 0; n < kPairs; ++n) {
                f16x8 hi, lo;
                load_x(n, hi, lo);
                add_x(n, hi, lo);
            }
        }
        border<0>();
#pragma unroll
        for (int k = 0; k < FM / 2; ++k) read_p(0, 0, k);
#pragma unroll
        for (int y = 0; y < FN; ++y) read_q(0, 0, y);
        // The products of one part; after each, its share of the next part's reads
        // and of the loads: a wave issues in order, and a burst of loads that the
        // memory path cannot take at once would hold up its products.
        auto multiply = [&](int h, int set, auto reads, auto loads, auto &&rd, auto &&ld) {
            constexpr int n = FM / 2 * FN, R = reads.value, L = loads.value;
#pragma unroll
            for (int k = 0; k < n; ++k) {
                const int x = k / FN, y = k % FN;
                f32x4 &c = acc[h * (FM / 2) + x][y];
                c = __builtin_amdgcn_mfma_f32_16x16x32_f16(p[h][x], q[set][y], c, 0, 0, 0);
                // the reads go first, so that the last have some products to land
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (r * (n - 2) / (R > 0 ? R : 1) == k) rd(r);
#pragma unroll
                for (int l = 0; l < L; ++l)
                    if ((2 * l + 1) * n / (2 * (L > 0 ? L : 1)) == k) ld(l);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        // One stage; set: its rows j.  No branch lies between a read of operands
        // and their use, so that the compiler waits for the older reads alone.
        auto stage = [&](auto wait, auto more, int set, int s) {
            constexpr int LP = more.value > 1 ? kLoadsP : 0, LQ = more.value > 1 ? kLoadsQ : 0;
            multiply(0, set, Int<FM / 2>{}, Int<LP>{}, [&](int k) { read_p(s, 1, k); },
                     [&](int k) { fill_p(s + NST - 1, k); });
            if constexpr (more.value > 0) border<wait.value>();
            multiply(1, set, Int<(more.value > 0 ? FM / 2 + FN : 0)>{}, Int<LQ>{},
                     [&](int k) {
                         // the first product's operands first
                         if (k == 0) read_p(s + 1, 0, 0);
                         else if (k <= FN) read_q(s + 1, set ^ 1, k - 1);
                         else read_p(s + 1, 0, k - FN);
                     },
                     [&](int k) { fill_q(s + NST - 1, k); });
        };
        constexpr int kLoads = kLoadsP + kLoadsQ;
        // loads younger than the next stage's: NST - 3 stages and this one's first
        constexpr Int<kLoads *(NST - 3) + kLoadsP> kWait{};
        int s = 0;
        if constexpr (kSpread) {
            if (spread) {
#pragma unroll
                for (int t = 0; t < kTurns; ++t) {
                    f16x8 hi[2], lo[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) load_x(2 * t + k, hi[k], lo[k]);
                    const int end = (steps - NST) / 2 * (t + 1) / kTurns * 2;
                    do {
                        stage(kWait, Int<2>{}, 0, s);
                        stage(kWait, Int<2>{}, 1, s + 1);
                        s += 2;
                    } while (s < end);
#pragma unroll
                    for (int k = 0; k < 2; ++k) add_x(2 * t + k, hi[k], lo[k]);
                }
            }
        }
        for (; s + NST < steps; s += 2) {
            stage(kWait, Int<2>{}, 0, s);
            stage(kWait, Int<2>{}, 1, s + 1);
        }
        // the last four: one more to load, two with a border, the last
        stage(kWait, Int<2>{}, 0, s);
        stage(Int<kLoads>{}, Int<1>{}, 1, s + 1);
        stage(Int<0>{}, Int<1>{}, 0, s + 2);
        stage(Int<0>{}, Int<0>{}, 1, s + 3);
    }
    if constexpr (KIND == kGramPart) {
        f32x4 *part = reinterpret_cast<f32x4 *>(at(ws, M.sums)) +
                      static_cast<int64_t>(tl.part) * (BM * BN / 4) + threadIdx.x;
#pragma unroll
        for (int x = 0; x < FM; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y) part[(x * FN + y) * 64 * WAVES] = acc[x][y];
        return;
    }

    // Epilogue, block by block of 32 x 32.  For b = 0, 1 this lane has column
    // colb(b) and, in v[b], the rows 8 g .. + 8 (X X^T: 4 g .. + 4 of either
    // half of the rows).
    lds_char *st = lds + wave * 2048;
    if constexpr (kSym || KIND == kLast) border<0>();
    const float phi = when & kFirst ? sc.phi0 : sc.phi, rho = when & kFirst ? sc.rho : 1.0f;
    const float alpha = kXXT   ? ldexpf(phi * phi, kLogA)
                        : KIND == kPoly ? ldexpf(coef.c, -kLogA)
                                        : ldexpf(rho, -kLogA);
    const bool vec = KIND == kLast && (lo32(M.out) & 15u) == 0 && (M.cols & 7) == 0;
#pragma unroll
    for (int x = 0; x < FM; x += 2)
#pragma unroll
        for (int y = 0; y < FN; y += 2) {
            const int ib = i0 + wm * WTM + x * 16, jb = j0 + wn * WTN + y * 16;
            if (ib >= M.mp || jb >= (kSym ? M.mp : M.np)) continue;
            Half8 v[2];
            int col[2], row[2];         // of the block; rows: of the first and second four
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                col[b] = kXXT ? 16 * b + (lane & 15) : perm_row(lane & 15, b);
                row[b] = kXXT ? 16 * b + 4 * g : 8 * g + 4 * b;
            }
            char *C = at(ws, kXXT ? M.a : M.b), *CL = at(ws, kXXT ? M.al : M.bl);
            Half8 low[2];               // of A and B
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = alpha * acc[x + (e >> 2)][y + b][e & 3];
                const int64_t o = panel_at(kSym ? M.mp : M.np, jb + col[b], ib + row[0]);
                auto halves = [&](f16x8 &hi, f16x8 &lo) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float f = settled(t[e]);
                        hi[e] = static_cast<_Float16>(f);
                        lo[e] = static_cast<_Float16>(f - static_cast<float>(hi[e]));
                    }
                };
                if constexpr (kXXT) {
                    auto put = [&](char *to, const Half8 &h) {
                        s16x4 *c = reinterpret_cast<s16x4 *>(to) + (o >> 2);
                        c[0] = h.q[0];
                        c[4] = h.q[1];
                    };
                    if constexpr (kFine) {
                        halves(v[b].f, low[b].f);
                        put(CL, low[b]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[b].f[e] = static_cast<_Float16>(t[e]);
                    }
                    put(C, v[b]);
                } else if constexpr (KIND == kPoly) {
                    const f16x8 old = reinterpret_cast<const f16x8 *>(at(ws, M.a))[o >> 3];
                    if constexpr (kFine) {
                        const f16x8 rest = reinterpret_cast<const f16x8 *>(at(ws, M.al))[o >> 3];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            t[e] = coef.b * (static_cast<float>(old[e]) + static_cast<float>(rest[e])) +
                                   t[e];
                        halves(v[b].f, low[b].f);
                        reinterpret_cast<f16x8 *>(CL)[o >> 3] = low[b].f;
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[b].f[e] =
                                static_cast<_Float16>(coef.b * static_cast<float>(old[e]) + t[e]);
                    }
                    reinterpret_cast<f16x8 *>(C)[o >> 3] = v[b].f;
                } else if constexpr (KIND == kApply) {
                    f16x8 lo;
                    halves(v[b].f, lo);
                    reinterpret_cast<f16x8 *>(at(ws, src ? M.t[0] : M.t[1]))[o >> 3] = v[b].f;
                    // other blocks read all of a low part that is an operand
                    reinterpret_cast<f16x8 *>(at(ws, kFine && !src ? M.lo2 : M.lo))[o >> 3] = lo;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[b].s[e] = static_cast<short>(to_bf16(t[e] * sc.phi));
                }
            }
            // the block turned over, through 2 KB of LDS: row ib + (lane & 31), its
            // columns 16 t + 8 (lane >> 5) .. + 8 in v[t]
            auto turn = [&](Half8(&v)[2]) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        *(lds_s16x4 *)(st + col[b] * 64 + row[c] * 2) = v[b].q[c];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    lds_char *a = st + (16 * t + 8 * (lane >> 5) + ((lane >> 2) & 3)) * 64 +
                                  (g & 1) * 32 + (lane & 3) * 8;
                    v[t].q[0] = read_tr(a);
                    v[t].q[1] = read_tr(a + 4 * 64);
                }
            };
            if ((kSym && tl.ti != tl.tj) || (KIND == kLast && M.wide)) turn(v);
            const int tr = ib + (lane & 31);
            if constexpr (kSym) {
                // a tile off the diagonal is its mirror image's values too
                if (tl.ti != tl.tj) {
                    auto mirror = [&](char *to, const Half8(&v)[2]) {
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            reinterpret_cast<f16x8 *>(
                                to)[panel_at(M.mp, tr, jb + 16 * t + 8 * (lane >> 5)) >> 3] = v[t].f;
                    };
                    mirror(C, v);
                    if constexpr (kFine) {
                        turn(low);
                        mirror(CL, low);
                    }
                }
            } else if constexpr (KIND == kLast) {
                // the row and the first of 8 neighbouring columns of the output
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int r = M.wide ? tr : jb + col[t];
                    const int c = M.wide ? jb + 16 * t + 8 * (lane >> 5) : ib + 8 * g;
                    if (r < M.rows && c < M.cols)
                        store_out(M.out + static_cast<int64_t>(r) * M.cols + c, v[t], M.cols - c,
                                  vec);
                }
            }
        }
}

// ---------------------------------------------------------------------------
// matrices with few rows
// ---------------------------------------------------------------------------

// Up to kSmallMax rows a block holds all m rows of a slab of NB columns of X in
// LDS and goes through the iteration by itself: with one slab the whole
// orthogonalisation is one launch, with more each iteration is one (its
// block sums the slabs' X X^T, makes B, multiplies its slab and leaves its part
// of the next X X^T), and a second one where there are too many parts to sum in
// every block.
//
// Every operand is taken as a high and a low fp16 part (three products of the
// four), to 2^-22: with few rows the roundings of A, of B and of X in the
// products are few and do not average out (fp16 alone was up to 5e-3 off with
// one to four rows), and the products are too small to bound the time.

template <int MP>
struct Small {
    static constexpr int NB = small_slab(MP);           // columns of a slab, at most
    static constexpr int nb = MP / 16;                  // 16 x 16 blocks a side
    static constexpr int kThreads = small_threads(MP), kWaves = kThreads / 64;
    // 16 x 16 blocks of A and B that one wave has
    static constexpr int kBJ = MP == 128 ? 4 : MP == 64 ? 2 : 1;
    // up to 64 rows a wave sums 32 x 32 of A over one stretch in kStretches
    static constexpr int kStretches = MP == 32 ? 8 : MP == 64 ? 2 : 1;
    static constexpr int kImage = NB * MP * 2;          // bytes of one part of X
    // in LDS the low part lies half of the banks further than the high one, so that
    // a lane's 8 bytes of either, one instruction, are not in the same banks
    static constexpr int kT = kImage + 128, kA = MP * MP * 2 + 128;
    // With 128 rows a wave has 32 x 32 of the upper half of A and B, which are
    // symmetric: ten waves, and the reads of LDS, which bound it, are half of those
    // of 16 waves with 16 x 64 of all (128 x 128: 43.8 -> 40.6 us).
    static constexpr bool kUpper = MP == 128;
    // those sums have LDS of their own: no barrier before A takes their place
    static constexpr int kLds = 2 * kT + 2 * kA + (MP == 128 ? 0 : kWaves * 4096);
};

// Element (row, col .. + 4 or 8) in LDS panels of 32 columns with `rows` rows; a
// row's 16-byte chunk sits at its index xor a number that the row's place among
// four fours gives: 0, 3, 2, 1.  Reads along rows of 16 bytes a lane, the products'
// results of 8 bytes in 16 rows and the transposing reads below all spread over the
// 64 banks then (with 0, 0, 2, 2 a quarter of all LDS cycles were conflicts, with
// 0, 2, 1, 3 those of the reads along rows).
__device__ __forceinline__ int small_at(int rows, int row, int col) {
    return (col >> 5) * rows * 64 + row * 64 +
           ((((col >> 3) & 3) ^ (-(row >> 2) & 3)) * 16) + (col & 7) * 2;
}

// Of the rows from row0, a multiple of 16, and the panel of column col0: what all
// lanes add to the place of a row and a column counted from there.
__device__ __forceinline__ int small_block(int rows, int row0, int col0) {
    return (col0 >> 5) * rows * 64 + row0 * 64;
}

// Place of this lane's four of a result: rows row0 .. + 16, columns col0 .. + 16.
__device__ __forceinline__ int small_four(int rows, int row0, int col0, int lane) {
    return small_block(rows, row0, col0) +
           small_at(rows, lane & 15, (col0 & 16) + 4 * (lane >> 4));
}

// Operand: 16 rows from row0, 32 columns from col0.
__device__ __forceinline__ f16x8 small_rows(const lds_char *t, int rows, int row0, int col0,
                                            int lane) {
    return *(const lds_f16x8 *)(t + small_block(rows, row0, col0) +
                                small_at(rows, lane & 15, 8 * (lane >> 4)));
}

// Operand: 16 columns from col0, 32 rows (the sum) from row0.
__device__ __forceinline__ f16x8 small_cols(lds_char *t, int rows, int row0, int col0, int lane) {
    const int k = (lane >> 4) * 8 + ((lane >> 2) & 3), col = (col0 & 16) + (lane & 3) * 4;
    t += small_block(rows, row0, col0);
    union {
        s16x4 s[2];
        f16x8 v;
    } u;
    u.s[0] = read_tr(t + small_at(rows, k, col));
    u.s[1] = read_tr(t + small_at(rows, k + 4, col));
    return u.v;
}

// c += (ph + pl) (qh + ql) without pl ql
__device__ __forceinline__ f32x4 fine_product(f16x8 ph, f16x8 pl, f16x8 qh, f16x8 ql, f32x4 c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, ql, c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(pl, qh, c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(ph, qh, c, 0, 0, 0);
}

// Four neighbouring values as high and low parts at byte offset o of hi and lo.
// (A factor that the compiler does not see the value of: the differences are then
// one instruction each that reads the half itself.)
__device__ __forceinline__ void put_split(lds_char *hi, lds_char *lo, int o, f32x4 x) {
    const float minus = settled(-1.0f);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = settled(x[e]);
    const f16x4 h = __builtin_convertvector(x, f16x4);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __builtin_fmaf(static_cast<float>(h[e]), minus, x[e]);
    *(lds_f16x4 *)(hi + o) = h;
    *(lds_f16x4 *)(lo + o) = __builtin_convertvector(x, f16x4);
}

template <int MP, bool kF32>
__global__ __launch_bounds__(Small<MP>::kThreads) void ortho_small_kernel(
    const OrthoTile *__restrict__ tiles, const OrthoMat *__restrict__ mats, void *ws, int32_t mode,
    int32_t step, int32_t n_steps, const OrthoCoef *__restrict__ coefs, double eps, int32_t growth) {
    using S = Small<MP>;
    constexpr int NB = S::NB, nb = S::nb, kBJ = S::kBJ, kSmallBlock = S::kThreads;
    __shared__ __attribute__((aligned(1024))) char smem[S::kLds];
    __shared__ double sums[S::kWaves];
    lds_char *th = (lds_char *)smem, *tlo = th + S::kT, *ah = tlo + S::kT, *al = ah + S::kA;
    f32x4 *scratch = reinterpret_cast<f32x4 *>(smem + 2 * S::kT + 2 * S::kA);

    const OrthoTile tl = tiles[blockIdx.x];
    const OrthoMat M = mats[tl.mat];
    const int tid = threadIdx.x;
    int lane = tid & 63;
    // nothing that follows from the lane is kept from one phase to the next: all their
    // addresses together do not fit the registers of 16 waves
    auto phase = [&]() {
        if constexpr (MP == 128) asm volatile("" : "+v"(lane));
    };
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slab = tl.ti, j0 = slab * M.slab;
    const int rows = M.n - j0 < M.slab ? M.n - j0 : M.slab, rows32 = (rows + 31) & ~31;
    // This wave's blocks of A and B, number y: block row bi + (y >> 1) and block column
    // bj + (y & 1) of the upper half's 32 x 32, otherwise bi and bj + y.
    int bi, bj;
    if constexpr (S::kUpper) {
        // 0 .. 9: rows 0 0 0 0 1 1 1 2 2 3, columns 0 1 2 3 1 2 3 2 3 3
        const int r = (wave >= 4) + (wave >= 7) + (wave >= 9);
        bi = 2 * r;
        bj = 2 * (wave - r * (7 - r) / 2);
    } else {
        bi = MP == 32 ? (wave >> 1) & 1 : wave >> 1;
        bj = (wave & 1) * kBJ;
    }
    auto row_of = [&](int y) { return (S::kUpper ? bi + (y >> 1) : bi) * 16; };
    auto col_of = [&](int y) { return (S::kUpper ? bj + (y & 1) : bj + y) * 16; };
    const bool mine = S::kUpper ? wave < 10 : MP > 32 || wave < 4;
    char *image = at(ws, M.t[0]) + static_cast<int64_t>(slab) * 2 * S::kImage;

    OrthoScal sc;
    if (mode == kSmallAll || mode == kSmallStart) {
        // eight neighbouring rows i of one column j a thread and turn; of a wide U a
        // wave takes 16 columns and 32 rows, whose 1 KB in LDS is of one piece
        auto wide_j = [](int u) { return (u >> 6) % (NB / 16) * 16 + (u & 15); };
        auto wide_i = [](int u) { return (u >> 6) / (NB / 16) * 4 + ((u >> 4) & 3); };
        constexpr int kTurns = (NB * MP / 8 + kSmallBlock - 1) / kSmallBlock;
        // every load leaves before the first is waited for: no branch around them,
        // places outside U read its first element instead
        float x[kTurns][8];
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
            const int u = t * kSmallBlock + tid;
            const int j = M.wide ? wide_j(u) : u / (MP / 8);
            const int i = (M.wide ? wide_i(u) : u % (MP / 8)) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t o = M.wide ? static_cast<int64_t>(i + e) * M.cols + j0 + j
                                         : static_cast<int64_t>(j0 + j) * M.cols + i + e;
                x[t][e] = load_in<kF32>(M.in, j < rows && i + e < M.m ? o : 0);
            }
        }
        double s = 0.0;
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
            const int u = t * kSmallBlock + tid;
            const int j = M.wide ? wide_j(u) : u / (MP / 8);
            const int i = (M.wide ? wide_i(u) : u % (MP / 8)) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[t][e] = j < rows && i + e < M.m ? x[t][e] : 0.0f;
                s += static_cast<double>(x[t][e]) * x[t][e];
            }
        }
        if (mode == kSmallStart) {
            s = 0.0;
            const double *parts = reinterpret_cast<const double *>(at(ws, M.parts));
            for (int i = tid; i < M.n_parts; i += kSmallBlock) s += parts[i];
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
        if (lane == 0) sums[wave] = s;
        __syncthreads();
        s = 0.0;
#pragma unroll
        for (int w = 0; w < S::kWaves; ++w) s += sums[w];
        int k;
        sc = scalars(sqrt(s), eps, growth, &k);
        const bool fine = sc.phi0 == sc.phi0 || isfinite(s);
        if (mode == kSmallStart && slab == 0 && tid == 0)
            *reinterpret_cast<OrthoScal *>(at(ws, M.scal)) = sc;
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
            const int u = t * kSmallBlock + tid;
            const int j = M.wide ? wide_j(u) : u / (MP / 8);
            const int i = (M.wide ? wide_i(u) : u % (MP / 8)) * 8;
            if (j < rows32 && i < MP) {
                Half8 h, l;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float f = fine ? settled(ldexpf(x[t][e], k)) : 0.0f;
                    h.f[e] = static_cast<_Float16>(f);
                    l.f[e] = static_cast<_Float16>(f - static_cast<float>(h.f[e]));
                }
                const int o = small_at(NB, j, i);
                *(lds_f16x8 *)(th + o) = h.f;
                *(lds_f16x8 *)(tlo + o) = l.f;
            }
        }
    } else {
        sc = *reinterpret_cast<const OrthoScal *>(at(ws, M.scal));
        // the slab as it was left: whole panels' rows
        for (int q = 0; q < MP / 32; ++q)
            for (int o = tid * 16; o < rows32 * 64; o += kSmallBlock * 16) {
                const int at16 = q * NB * 64 + o;
                *reinterpret_cast<u32x4 *>(smem + at16) =
                    *reinterpret_cast<const u32x4 *>(image + at16);
                *reinterpret_cast<u32x4 *>(smem + S::kT + at16) =
                    *reinterpret_cast<const u32x4 *>(image + S::kImage + at16);
            }
    }
    __syncthreads();

    f32x4 a[kBJ];
    // this wave's blocks of X X^T over the slab
    auto gram = [&]() {
        if constexpr (S::kStretches > 1) {
            const int quad = MP == 64 ? wave & 3 : 0, qi = (quad >> 1) * 32, qj = (quad & 1) * 32;
            const int stretch = MP == 64 ? wave >> 2 : wave;
            f32x4 c[2][2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) c[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
            for (int r = stretch * 32; r < rows32; r += 32 * S::kStretches) {
                f16x8 ph[2], pl[2], qh[2], ql[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    ph[x] = small_cols(th, NB, r, qi + 16 * x, lane);
                    pl[x] = small_cols(tlo, NB, r, qi + 16 * x, lane);
                    qh[x] = small_cols(th, NB, r, qj + 16 * x, lane);
                    ql[x] = small_cols(tlo, NB, r, qj + 16 * x, lane);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        c[x][y] = fine_product(ph[x], pl[x], qh[y], ql[y], c[x][y]);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) scratch[(wave * 4 + x * 2 + y) * 64 + lane] = c[x][y];
            __syncthreads();
            // the stretches in order
#pragma unroll
            for (int y = 0; y < kBJ; ++y) {
                const int k = bj + y, of = (bi >> 1) * 2 + (k >> 1), sub = (bi & 1) * 2 + (k & 1);
                a[y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int t = 0; t < S::kStretches; ++t)
                    if (32 * t < rows32)
                        a[y] += scratch[((MP == 64 ? t * 4 + of : t) * 4 + sub) * 64 + lane];
            }
        } else {
#pragma unroll
            for (int y = 0; y < kBJ; ++y) a[y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (!mine) return;
            for (int r = 0; r < rows32; r += 32) {
                f16x8 ph[2], pl[2], qh[2], ql[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    ph[x] = small_cols(th, NB, r, (bi + x) * 16, lane);
                    pl[x] = small_cols(tlo, NB, r, (bi + x) * 16, lane);
                    qh[x] = small_cols(th, NB, r, (bj + x) * 16, lane);
                    ql[x] = small_cols(tlo, NB, r, (bj + x) * 16, lane);
                }
#pragma unroll
                for (int y = 0; y < kBJ; ++y)
                    a[y] = fine_product(ph[y >> 1], pl[y >> 1], qh[y & 1], ql[y & 1], a[y]);
            }
        }
    };
    // parts of A: one 16 x 16 block after the other, a lane's four values together
    constexpr int kPart = small_part(MP);
    auto part = [&](int k, int y) {
        return reinterpret_cast<f32x4 *>(at(ws, (k & 1) ? M.b : M.a)) +
               (S::kUpper ? wave * 4 + y : bi * nb + bj + y) * 64 + lane;
    };
    // this wave's blocks, in t by rows of the second index, to their other half
    auto mirror = [&](lds_char *t) {
        if constexpr (S::kUpper) {
            if (bi == bj) return;
#pragma unroll
            for (int x = 0; x < 2; ++x)
                *(lds_f16x8 *)(t + small_block(MP, (bi + x) * 16, bj * 16) +
                               small_at(MP, lane & 15, 8 * (lane >> 4))) =
                    small_cols(t, MP, bj * 16, (bi + x) * 16, lane);
        }
    };
    if (mode == kSmallAll || mode == kSmallStart) gram();
    if (mode == kSmallStart && mine) {
#pragma unroll
        for (int y = 0; y < kBJ; ++y) part(0, y)[static_cast<int64_t>(slab) * kPart] = a[y];
    }
    const int from = mode == kSmallAll ? 0 : step;
    const int to = mode == kSmallAll ? n_steps : mode == kSmallStart ? 0 : step + 1;
    for (int k = from; k < to; ++k) {
        const OrthoCoef c = coefs[k];
        phase();
        if (mode != kSmallAll && mine) {
            // the parts' sum, in order; eight loads of a lane under way
            constexpr int kAhead = 8 / kBJ;
#pragma unroll
            for (int y = 0; y < kBJ; ++y) a[y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            for (int t = 0; t < M.n_sums; t += kAhead) {
                f32x4 v[kAhead][kBJ];
#pragma unroll
                for (int x = 0; x < kAhead; ++x)
#pragma unroll
                    for (int y = 0; y < kBJ; ++y)
                        v[x][y] = part(k, y)[static_cast<int64_t>(t + x < M.n_sums ? t + x : t) * kPart];
#pragma unroll
                for (int x = 0; x < kAhead; ++x)
#pragma unroll
                    for (int y = 0; y < kBJ; ++y)
                        if (t + x < M.n_sums) a[y] += v[x][y];
            }
        }
        const float phi = k == 0 ? sc.phi0 : sc.phi, rho = k == 0 ? sc.rho : 1.0f;
        // A, scaled, as operands: a block's four rows a lane as columns (A is symmetric)
        const float alpha = ldexpf(phi * phi, kLogA);
        f32x4 av[kBJ];
        if (mine) {
#pragma unroll
            for (int y = 0; y < kBJ; ++y) {
#pragma unroll
                for (int e = 0; e < 4; ++e) av[y][e] = alpha * a[y][e];
                put_split(ah, al, small_four(MP, col_of(y), row_of(y), lane), av[y]);
            }
            mirror(ah);
            mirror(al);
        }
        __syncthreads();
        f32x4 b[kBJ];
        if (mine) {
#pragma unroll
            for (int y = 0; y < kBJ; ++y) b[y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < MP; q += 32) {
                constexpr int kP = S::kUpper ? 2 : 1, kQ = kBJ / kP;
                f16x8 ph[kP], pl[kP], qh[kQ], ql[kQ];
#pragma unroll
                for (int x = 0; x < kP; ++x) {
                    ph[x] = small_rows(ah, MP, (bi + x) * 16, q, lane);
                    pl[x] = small_rows(al, MP, (bi + x) * 16, q, lane);
                }
#pragma unroll
                for (int x = 0; x < kQ; ++x) {
                    qh[x] = small_rows(ah, MP, (bj + x) * 16, q, lane);
                    ql[x] = small_rows(al, MP, (bj + x) * 16, q, lane);
                }
#pragma unroll
                for (int y = 0; y < kBJ; ++y)
                    b[y] = fine_product(ph[y / kQ], pl[y / kQ], qh[y % kQ], ql[y % kQ], b[y]);
            }
        }
        __syncthreads();
        if (mine) {
            const float cc = ldexpf(c.c, -kLogA);
#pragma unroll
            for (int y = 0; y < kBJ; ++y) {
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = c.b * av[y][e] + cc * b[y][e];
                put_split(ah, al, small_four(MP, col_of(y), row_of(y), lane), v);
            }
            mirror(ah);
            mirror(al);
        }
        __syncthreads();
        phase();
        // X = a X + B X: a wave takes 16 columns j at a time, which no other wave reads or writes
        const bool last = k + 1 == n_steps;
        const float ca = ldexpf(c.a, kLogA), cb = ldexpf(rho, -kLogA);
        // up to 64 rows B's operands stay in registers
        constexpr bool kHeld = MP <= 64;
        f16x8 ph[kHeld ? nb : 1][kHeld ? MP / 32 : 1], pl[kHeld ? nb : 1][kHeld ? MP / 32 : 1];
        if constexpr (kHeld) {
#pragma unroll
            for (int x = 0; x < nb; ++x)
#pragma unroll
                for (int q = 0; q < MP / 32; ++q) {
                    ph[x][q] = small_rows(ah, MP, x * 16, q * 32, lane);
                    pl[x][q] = small_rows(al, MP, x * 16, q * 32, lane);
                }
        }
        // a tall matrix's fours of a row in one store where they lie at 8 bytes
        const bool quads = !M.wide && (M.cols & 3) == 0 && (lo32(M.out) & 7u) == 0;
        // with 128 rows two waves share 16 columns, half of the rows each
        constexpr int kSide = kHeld ? 1 : 2, kX = nb / kSide;
        const int x0 = kHeld ? 0 : (wave & 1) * kX;
        static_assert(kHeld || NB == S::kWaves / kSide * 16, "one turn");
        for (int r = wave / kSide * 16; r < (kHeld ? rows : NB); r += S::kWaves / kSide * 16) {
            f16x8 qh[MP / 32], ql[MP / 32];
#pragma unroll
            for (int q = 0; q < MP / 32; ++q) {
                qh[q] = small_rows(th, NB, r, q * 32, lane);
                ql[q] = small_rows(tlo, NB, r, q * 32, lane);
            }
            if constexpr (!kHeld) __syncthreads();      // both have read them
            const int j = r + (lane & 15);
            // kAt blocks of rows at a time, whose products do not wait for each other: all
            // of them, or one where the registers hold no more beside the column's
            constexpr int kAt = kHeld ? kX : 1;
#pragma unroll
            for (int xs = 0; xs < kX; xs += kAt) {
                f32x4 v[kAt];
#pragma unroll
                for (int y = 0; y < kAt; ++y) {
                    const int o = small_four(NB, r, (x0 + xs + y) * 16, lane);
                    const f16x4 xh = *(lds_f16x4 *)(th + o), xl = *(lds_f16x4 *)(tlo + o);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[y][e] = __builtin_fmaf(
                            static_cast<float>(xh[e]), ca,
                            __builtin_fmaf(static_cast<float>(xl[e]), ca, 0.0f));
                }
#pragma unroll
                for (int q = 0; q < MP / 32; ++q) {
                    f16x8 h[kAt], l[kAt];
#pragma unroll
                    for (int y = 0; y < kAt; ++y) {
                        if constexpr (kHeld) {
                            h[y] = ph[xs + y][q];
                            l[y] = pl[xs + y][q];
                        } else {
                            h[y] = small_rows(ah, MP, (x0 + xs + y) * 16, q * 32, lane);
                            l[y] = small_rows(al, MP, (x0 + xs + y) * 16, q * 32, lane);
                        }
                    }
#pragma unroll
                    for (int y = 0; y < kAt; ++y)
                        v[y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(h[y], ql[q], v[y], 0, 0, 0);
#pragma unroll
                    for (int y = 0; y < kAt; ++y)
                        v[y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(l[y], qh[q], v[y], 0, 0, 0);
#pragma unroll
                    for (int y = 0; y < kAt; ++y)
                        v[y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(h[y], qh[q], v[y], 0, 0, 0);
                }
                if (!last) {
                    if (kHeld || r < rows) {
#pragma unroll
                        for (int y = 0; y < kAt; ++y) {
                            f32x4 w;
#pragma unroll
                            for (int e = 0; e < 4; ++e) w[e] = cb * v[y][e];
                            put_split(th, tlo, small_four(NB, r, (x0 + xs + y) * 16, lane), w);
                        }
                    }
                } else if (j < rows) {
#pragma unroll
                    for (int y = 0; y < kAt; ++y) {
                        const int i = (x0 + xs + y) * 16 + 4 * (lane >> 4);
                        uint16_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = to_bf16(cb * v[y][e] * sc.phi);
                        uint16_t *at = M.out + (M.wide ? static_cast<int64_t>(i) * M.cols + j0 + j
                                                       : static_cast<int64_t>(j0 + j) * M.cols + i);
                        if (quads && i < M.m) {
                            *reinterpret_cast<u32x2 *>(at) =
                                u32x2{static_cast<uint32_t>(w[0]) | (static_cast<uint32_t>(w[1]) << 16),
                                      static_cast<uint32_t>(w[2]) | (static_cast<uint32_t>(w[3]) << 16)};
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (i + e < M.m)
                                    at[e * (M.wide ? static_cast<int64_t>(M.cols) : 1)] = w[e];
                        }
                    }
                }
            }
        }
        __syncthreads();
        if (last) break;
        phase();
        gram();
        if (mode == kSmallStep && mine) {
#pragma unroll
            for (int y = 0; y < kBJ; ++y)
                part(k + 1, y)[static_cast<int64_t>(slab) * kPart] = a[y];
        }
    }
    if (mode == kSmallStart || mode == kSmallStep) {
        __syncthreads();
        for (int q = 0; q < MP / 32; ++q)
            for (int o = tid * 16; o < rows32 * 64; o += kSmallBlock * 16) {
                const int at16 = q * NB * 64 + o;
                *reinterpret_cast<u32x4 *>(image + at16) =
                    *reinterpret_cast<const u32x4 *>(smem + at16);
                *reinterpret_cast<u32x4 *>(image + S::kImage + at16) =
                    *reinterpret_cast<const u32x4 *>(smem + S::kT + at16);
            }
    }
}

// Sums the parts of A of the matrices that have too many for every block to sum
// them: the sum replaces the first part.
__global__ __launch_bounds__(kBlock) void ortho_sums_kernel(const OrthoTile *__restrict__ tiles,
                                                            const OrthoMat *__restrict__ mats,
                                                            void *ws, int32_t step) {
    const OrthoTile tl = tiles[blockIdx.x];
    const OrthoMat M = mats[tl.mat];
    const int64_t size = small_part(M.mp);
    f32x4 *p = reinterpret_cast<f32x4 *>(at(ws, (step & 1) ? M.b : M.a)) + tl.ti * kBlock +
               threadIdx.x;
    f32x4 v = p[0];
#pragma unroll 8
    for (int t = 1; t < tl.tj; ++t) v += p[t * size];
    p[0] = v;
}

}  // namespace

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------

hipError_t launch_ortho_norm(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             bool f32, hipStream_t st) {
    if (n == 0) return hipSuccess;
    if (f32) ortho_norm_kernel<true><<<static_cast<unsigned>(n), kBlock, 0, st>>>(tiles, mats, ws);
    else ortho_norm_kernel<false><<<static_cast<unsigned>(n), kBlock, 0, st>>>(tiles, mats, ws);
    return hipGetLastError();
}

hipError_t launch_ortho_init(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             bool f32, double eps, int32_t growth, hipStream_t st) {
    if (n == 0) return hipSuccess;
    if (f32)
        ortho_init_kernel<true><<<static_cast<unsigned>(n), kBlock, 0, st>>>(tiles, mats, ws, eps,
                                                                             growth);
    else
        ortho_init_kernel<false><<<static_cast<unsigned>(n), kBlock, 0, st>>>(tiles, mats, ws, eps,
                                                                              growth);
    return hipGetLastError();
}

namespace {

template <int KIND, bool kFine>
hipError_t launch_tiles(int32_t tile, const OrthoTile *tiles, int64_t n, const OrthoMat *mats,
                          void *ws, int32_t src, int32_t when, int32_t split, OrthoCoef c,
                          hipStream_t st) {
    if (n == 0) return hipSuccess;
    const unsigned grid = static_cast<unsigned>(n);
    if (tile == 256)
        ortho_product_kernel<KIND, 256, 256, 2, 4, kFine>
            <<<grid, product_threads(256), 0, st>>>(tiles, mats, ws, src, when, split, c);
    else if (tile == 192)
        ortho_product_kernel<KIND, 192, 192, 6, 2, kFine>
            <<<grid, product_threads(192), 0, st>>>(tiles, mats, ws, src, when, split, c);
    else if (tile == 128)
        ortho_product_kernel<KIND, 128, 128, 2, 2, kFine>
            <<<grid, product_threads(128), 0, st>>>(tiles, mats, ws, src, when, split, c);
    else if (tile == 64)
        ortho_product_kernel<KIND, 64, 64, 2, 2, kFine>
            <<<grid, product_threads(64), 0, st>>>(tiles, mats, ws, src, when, split, c);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

template <int KIND>
hipError_t launch_product(int32_t tile, const OrthoTile *tiles, int64_t n, const OrthoMat *mats,
                          void *ws, int32_t src, int32_t when, int32_t split, OrthoCoef c,
                          hipStream_t st) {
    if (tile & kTileFine)
        return launch_tiles<KIND, true>(tile & ~kTileFine, tiles, n, mats, ws, src, when, split, c, st);
    return launch_tiles<KIND, false>(tile, tiles, n, mats, ws, src, when, split, c, st);
}

}  // namespace

namespace {

template <bool kF32>
void small(int32_t mp, unsigned n, const OrthoTile *tiles, const OrthoMat *mats, void *ws,
           int32_t mode, int32_t step, int32_t n_steps, const OrthoCoef *coefs, double eps,
           int32_t growth, hipStream_t st) {
    if (mp == 32)
        ortho_small_kernel<32, kF32><<<n, Small<32>::kThreads, 0, st>>>(tiles, mats, ws, mode, step,
                                                                n_steps, coefs, eps, growth);
    else if (mp == 64)
        ortho_small_kernel<64, kF32><<<n, Small<64>::kThreads, 0, st>>>(tiles, mats, ws, mode, step,
                                                                n_steps, coefs, eps, growth);
    else
        ortho_small_kernel<128, kF32><<<n, Small<128>::kThreads, 0, st>>>(tiles, mats, ws, mode, step,
                                                                 n_steps, coefs, eps, growth);
}

}  // namespace

hipError_t launch_ortho_small(int32_t mp, const OrthoTile *tiles, int64_t n, const OrthoMat *mats,
                              void *ws, bool f32, int32_t mode, int32_t step, int32_t n_steps,
                              const OrthoCoef *coefs, double eps, int32_t growth, hipStream_t st) {
    if (n == 0) return hipSuccess;
    if (f32)
        small<true>(mp, static_cast<unsigned>(n), tiles, mats, ws, mode, step, n_steps, coefs, eps,
                    growth, st);
    else
        small<false>(mp, static_cast<unsigned>(n), tiles, mats, ws, mode, step, n_steps, coefs, eps,
                     growth, st);
    return hipGetLastError();
}

hipError_t launch_ortho_sums(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             int32_t step, hipStream_t st) {
    if (n == 0) return hipSuccess;
    ortho_sums_kernel<<<static_cast<unsigned>(n), kBlock, 0, st>>>(tiles, mats, ws, step);
    return hipGetLastError();
}

hipError_t launch_ortho_gram(int32_t tile, const OrthoTile *tiles, int64_t n,
                             const OrthoTile *join, int64_t n_join, int32_t split,
                             const OrthoMat *mats, void *ws, int32_t src, bool first,
                             hipStream_t st) {
    const int32_t when = first ? kFirst : 0;
    if (split == 1)
        return launch_product<kGram>(tile, tiles, n, mats, ws, src, when, 1, OrthoCoef{}, st);
    const hipError_t e =
        launch_product<kGramPart>(tile, tiles, n, mats, ws, src, when, split, OrthoCoef{}, st);
    if (e != hipSuccess) return e;
    return launch_product<kGramJoin>(tile, join, n_join, mats, ws, src, when, split, OrthoCoef{},
                                     st);
}

hipError_t launch_ortho_poly(int32_t tile, const OrthoTile *tiles, int64_t n, const OrthoMat *mats,
                             void *ws, OrthoCoef c, hipStream_t st) {
    return launch_product<kPoly>(tile, tiles, n, mats, ws, 0, 0, 1, c, st);
}

hipError_t launch_ortho_apply(int32_t tile, const OrthoTile *tiles, int64_t n,
                              const OrthoMat *mats, void *ws, int32_t src, bool first, bool high,
                              bool last, OrthoCoef c, hipStream_t st) {
    const int32_t when = (first ? kFirst : 0) | (high ? kHigh : 0);
    if (last) return launch_product<kLast>(tile, tiles, n, mats, ws, src, when, 1, c, st);
    return launch_product<kApply>(tile, tiles, n, mats, ws, src, when, 1, c, st);
}

}  // namespace fsdp
