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
// one of low rank (relative, in the 2-norm; bf16 1e-2 to 0.2).  The term a X
// therefore takes X as a high and a low fp16 part (22 bits); the products,
// which vanish with the singular value, take the high part.  That leaves 3e-4
// to 2e-3, below the 1.7e-3 of rounding the result to bf16 itself or near it.
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
typedef __attribute__((address_space(3))) f16x8 lds_f16x8;

// log2 of the scale of A and B
constexpr int kLogA = 11;
// log2 of the scale of X where the norm is not lost in eps
constexpr int kLogX = 12;

__device__ __forceinline__ char *at(void *ws, int64_t off) { return static_cast<char *>(ws) + off; }

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

// Sums of squares in fp64: no scaling is needed for the smallest and largest
// values, and the order is fixed.
template <bool kF32>
__global__ __launch_bounds__(kBlock) void ortho_norm_kernel(const OrthoTile *__restrict__ tiles,
                                                            const OrthoMat *__restrict__ mats,
                                                            void *ws) {
    const OrthoTile tl = tiles[blockIdx.x];
    const OrthoMat M = mats[tl.mat];
    const int64_t total = static_cast<int64_t>(M.rows) * M.cols;
    const int64_t per = (total + M.n_parts - 1) / M.n_parts;
    const int64_t lo = per * tl.ti, hi = lo + per < total ? lo + per : total;
    double s = 0.0;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kBlock) {
        const double x = load_in<kF32>(M.in, i);
        s += x * x;
    }
    s = block_sum(s);
    if (threadIdx.x == 0) reinterpret_cast<double *>(at(ws, M.parts))[tl.ti] = s;
}

// X^T's 64 x 64 piece (rows 64 tj of n, columns 64 ti of m).  Stored is U
// 2^k, exact in fp16 for bf16 inputs within 2^-26 of the norm (the low part
// holds the rest), where 2^k puts the norm at 2^kLogX or up to twice that.
template <bool kF32>
__global__ __launch_bounds__(kBlock) void ortho_init_kernel(const OrthoTile *__restrict__ tiles,
                                                            const OrthoMat *__restrict__ mats,
                                                            void *ws, double eps, int32_t growth) {
    __shared__ float buf[64][65];
    const OrthoTile tl = tiles[blockIdx.x];
    const OrthoMat M = mats[tl.mat];
    const double *parts = reinterpret_cast<const double *>(at(ws, M.parts));
    double s = 0.0;
    for (int i = threadIdx.x; i < M.n_parts; i += kBlock) s += parts[i];
    const double norm = sqrt(block_sum(s));
    // A norm that is not finite makes the scalars NaN and so every output; the
    // stored X is then zero.  X = U / (norm + eps) is small where eps
    // outweighs the norm: up to what the iterations can magnify it back, X is
    // scaled up instead.
    const bool fine = isfinite(norm);
    int e = 0, up = 0;
    float phi0 = __builtin_nanf(""), phi = 0.0f, rho = __builtin_nanf("");
    if (fine) {
        double p0 = eps > 0.0 ? 1.0 : phi0;       // X = stored * p0; zero / 0 is NaN
        if (norm > 0.0) {
            e = ilogb(norm);
            const double r = norm / (norm + eps);
            up = r > 0.0 ? -ilogb(r) - growth : 100;
            up = up < 0 ? 0 : (up > 100 ? 100 : up);
            p0 = 1.0 / ldexp(norm + eps, kLogX - e);
        }
        phi = ldexpf(1.0f, -(kLogX + up));
        phi0 = static_cast<float>(p0);
        rho = static_cast<float>(ldexp(p0, kLogX + up));
    }
    if (tl.ti == 0 && tl.tj == 0 && threadIdx.x == 0)
        *reinterpret_cast<OrthoScal *>(at(ws, M.scal)) = OrthoScal{phi0, phi, rho, 0.0f};
    const int k = kLogX - e;
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    const int r0 = (M.wide ? tl.ti : tl.tj) * 64, c0 = (M.wide ? tl.tj : tl.ti) * 64;
    for (int y = ty; y < 64; y += kBlock / 64) {
        const int r = r0 + y, c = c0 + tx;
        float x = 0.0f;
        if (fine && r < M.rows && c < M.cols)
            x = ldexpf(load_in<kF32>(M.in, static_cast<int64_t>(r) * M.cols + c), k);
        buf[y][tx] = x;
    }
    __syncthreads();
    _Float16 *hi = reinterpret_cast<_Float16 *>(at(ws, M.t[0]));
    _Float16 *lo = reinterpret_cast<_Float16 *>(at(ws, M.lo));
    for (int y = ty; y < 64; y += kBlock / 64) {
        const float x = M.wide ? buf[tx][y] : buf[y][tx];
        const _Float16 h = static_cast<_Float16>(x);
        const int64_t o = panel_at(M.np, tl.tj * 64 + y, tl.ti * 64 + tx);
        hi[o] = h;
        lo[o] = static_cast<_Float16>(x - static_cast<float>(h));
    }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

enum { kGram = 0, kPoly = 1, kApply = 2, kLast = 3 };

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

// Four rows of 16 columns: lane l of a 16-lane group reads 4 neighbouring
// columns (8 bytes at t) of row l >> 2, and gets column l of the 16 that lanes
// 0 to 3 read, of those 4 rows.  (restrict: with aliasing facts on the read the
// compiler does not wait for every load to LDS that is under way before it;
// the borders wait for those that matter.)
__device__ __forceinline__ s16x4 read_tr(lds_char *__restrict__ t) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)t);
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

// x as one fp32 value.  Without this the compiler may take a product and its
// conversion to fp16 as one operation of one rounding in one place and as two
// in another, and a high part that is stored then differs, where the two
// round apart, from the one that the low part was taken against.
__device__ __forceinline__ float settled(float x) {
    asm volatile("" : "+v"(x));
    return x;
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
template <int KIND, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM *WN) void ortho_product_kernel(
    const OrthoTile *__restrict__ tiles, const OrthoMat *__restrict__ mats, void *ws, int32_t src,
    int32_t first, OrthoCoef coef) {
    constexpr int WAVES = WM * WN, WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
    constexpr int NST = 4;
    constexpr bool kSym = KIND == kGram || KIND == kPoly;
    constexpr int kStage = (BM + BN) * kBK * 2, kLoadsP = BM / 16 / WAVES,
                  kLoadsQ = BN / 16 / WAVES;
    static_assert(BM % (16 * WAVES) == 0 && BN % (16 * WAVES) == 0, "whole loads per wave");
    static_assert(NST * kStage >= WAVES * 2048 && kBK == 32 && FM % 4 == 0 && FN % 2 == 0, "");
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

    // load k of this wave's kLoadsP of stage s's rows i, or of its kLoadsQ of the rows j
    auto fill_p = [&](int s, int k) {
        lds_char *b = lds + (s & (NST - 1)) * kStage;
        const int u = k * WAVES + wave;
        if constexpr (KIND == kGram) {
            // rows of X^T are the sum, columns i and j
            const uint32_t panel = static_cast<uint32_t>(M.np) * 64u;
            const int at = i0 / 32, n = M.mp / 32 - at < BM / 32 ? M.mp / 32 - at : BM / 32;
            fill_cols(b, T + static_cast<int64_t>(at) * panel, n * panel, panel, s, u, lane);
        } else {
            const char *A = at(ws, KIND == kPoly ? M.a : M.b);
            const int n = M.mp - i0 < BM ? M.mp - i0 : BM;
            fill_rows(b, A + (static_cast<int64_t>(s) * M.mp + i0) * 64, n * 64u, u, lane);
        }
    };
    auto fill_q = [&](int s, int k) {
        lds_char *b = lds + (s & (NST - 1)) * kStage + BM * 64;
        const int u = k * WAVES + wave;
        if constexpr (KIND == kGram) {
            const uint32_t panel = static_cast<uint32_t>(M.np) * 64u;
            const int at = j0 / 32, n = M.mp / 32 - at < BN / 32 ? M.mp / 32 - at : BN / 32;
            fill_cols(b, T + static_cast<int64_t>(at) * panel, n * panel, panel, s, u, lane);
        } else {
            const char *A = KIND == kPoly ? at(ws, M.a) : T;
            const int rq = KIND == kPoly ? M.mp : M.np, n = rq - j0 < BN ? rq - j0 : BN;
            fill_rows(b, A + (static_cast<int64_t>(s) * rq + j0) * 64, n * 64u, u, lane);
        }
    };
    f16x8 p[2][FM / 2], q[2][FN];
    // operand k of part h of stage s's rows i; of its rows j, into set `set`
    auto read_p = [&](int s, int h, int k) {
        lds_char *t = lds + (s & (NST - 1)) * kStage;
        const int x = h * (FM / 2) + k, base = wm * WTM + (x >> 1) * 32;
        if constexpr (KIND == kGram) p[h][k] = read_cols(t, base + (x & 1) * 16, lane);
        else p[h][k] = read_rows(t, base + perm_row(lane & 15, x & 1), lane);
    };
    auto read_q = [&](int s, int set, int y) {
        lds_char *t = lds + (s & (NST - 1)) * kStage + BM * 64;
        const int base = wn * WTN + (y >> 1) * 32;
        if constexpr (KIND == kGram) q[set][y] = read_cols(t, base + (y & 1) * 16, lane);
        else q[set][y] = read_rows(t, base + perm_row(lane & 15, y & 1), lane);
    };

    const int steps = (KIND == kGram ? M.np : M.mp) / kBK;       // a multiple of four
#pragma unroll
    for (int s = 0; s < NST - 1; ++s) {
#pragma unroll
        for (int k = 0; k < kLoadsP; ++k) fill_p(s, k);
#pragma unroll
        for (int k = 0; k < kLoadsQ; ++k) fill_q(s, k);
    }
    f32x4 acc[FM][FN];
    if constexpr (kSym) {
#pragma unroll
        for (int x = 0; x < FM; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    } else {
        // the sums start from a X, so that its loads overlap the first stages'
        const float ca = ldexpf(coef.a, kLogA);
#pragma unroll
        for (int x = 0; x < FM; x += 2)
#pragma unroll
            for (int y = 0; y < FN; ++y) {
                const int i = i0 + wm * WTM + x * 16 + 8 * g;
                const int j = j0 + wn * WTN + (y >> 1) * 32 + perm_row(lane & 15, y & 1);
                f16x8 hi{}, lo{};
                if (i < M.mp && j < M.np) {
                    const int64_t o = panel_at(M.np, j, i) >> 3;
                    hi = reinterpret_cast<const f16x8 *>(T)[o];
                    lo = reinterpret_cast<const f16x8 *>(at(ws, M.lo))[o];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[x + (e >> 2)][y][e & 3] =
                        ca * (static_cast<float>(hi[e]) + static_cast<float>(lo[e]));
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
    for (; s + NST < steps; s += 2) {
        stage(kWait, Int<2>{}, 0, s);
        stage(kWait, Int<2>{}, 1, s + 1);
    }
    // the last four: one more to load, two with a border, the last
    stage(kWait, Int<2>{}, 0, s);
    stage(Int<kLoads>{}, Int<1>{}, 1, s + 1);
    stage(Int<0>{}, Int<1>{}, 0, s + 2);
    stage(Int<0>{}, Int<0>{}, 1, s + 3);

    // Epilogue, block by block of 32 x 32.  For b = 0, 1 this lane has column
    // colb(b) and, in v[b], the rows 8 g .. + 8 (X X^T: 4 g .. + 4 of either
    // half of the rows).
    lds_char *st = lds + wave * 2048;
    if constexpr (kSym || KIND == kLast) border<0>();
    const float phi = first ? sc.phi0 : sc.phi, rho = first ? sc.rho : 1.0f;
    const float alpha = KIND == kGram   ? ldexpf(phi * phi, kLogA)
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
                col[b] = KIND == kGram ? 16 * b + (lane & 15) : perm_row(lane & 15, b);
                row[b] = KIND == kGram ? 16 * b + 4 * g : 8 * g + 4 * b;
            }
            char *C = at(ws, KIND == kGram ? M.a : M.b);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float t[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = alpha * acc[x + (e >> 2)][y + b][e & 3];
                const int64_t o = panel_at(kSym ? M.mp : M.np, jb + col[b], ib + row[0]);
                if constexpr (KIND == kGram) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[b].f[e] = static_cast<_Float16>(t[e]);
                    s16x4 *c = reinterpret_cast<s16x4 *>(C) + (o >> 2);
                    c[0] = v[b].q[0];
                    c[4] = v[b].q[1];
                } else if constexpr (KIND == kPoly) {
                    const f16x8 old = reinterpret_cast<const f16x8 *>(at(ws, M.a))[o >> 3];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[b].f[e] =
                            static_cast<_Float16>(coef.b * static_cast<float>(old[e]) + t[e]);
                    reinterpret_cast<f16x8 *>(C)[o >> 3] = v[b].f;
                } else if constexpr (KIND == kApply) {
                    f16x8 lo;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float f = settled(t[e]);
                        v[b].f[e] = static_cast<_Float16>(f);
                        lo[e] = static_cast<_Float16>(f - static_cast<float>(v[b].f[e]));
                    }
                    reinterpret_cast<f16x8 *>(at(ws, src ? M.t[0] : M.t[1]))[o >> 3] = v[b].f;
                    reinterpret_cast<f16x8 *>(at(ws, M.lo))[o >> 3] = lo;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[b].s[e] = static_cast<short>(bf16_rne(t[e] * sc.phi));
                }
            }
            // the block turned over, through 2 KB of LDS: row ib + (lane & 31), its
            // columns 16 t + 8 (lane >> 5) .. + 8 in v[t]
            if ((kSym && tl.ti != tl.tj) || (KIND == kLast && M.wide)) {
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
            }
            const int tr = ib + (lane & 31);
            if constexpr (kSym) {
                // a tile off the diagonal is its mirror image's values too
                if (tl.ti != tl.tj) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        reinterpret_cast<f16x8 *>(
                            C)[panel_at(M.mp, tr, jb + 16 * t + 8 * (lane >> 5)) >> 3] = v[t].f;
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

}  // namespace

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------

#ifndef FSDP_ORTHO_BM
#define FSDP_ORTHO_BM 128
#define FSDP_ORTHO_BN 128
#define FSDP_ORTHO_WM 2
#define FSDP_ORTHO_WN 2
#endif
#define TILE_ARGS FSDP_ORTHO_BM, FSDP_ORTHO_BN, FSDP_ORTHO_WM, FSDP_ORTHO_WN
#define TILE_THR (64 * FSDP_ORTHO_WM * FSDP_ORTHO_WN)

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

hipError_t launch_ortho_gram(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             int32_t src, bool first, hipStream_t st) {
    if (n == 0) return hipSuccess;
    ortho_product_kernel<kGram, TILE_ARGS><<<static_cast<unsigned>(n), TILE_THR, 0, st>>>(
        tiles, mats, ws, src, first, OrthoCoef{});
    return hipGetLastError();
}

hipError_t launch_ortho_poly(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             OrthoCoef c, hipStream_t st) {
    if (n == 0) return hipSuccess;
    ortho_product_kernel<kPoly, TILE_ARGS><<<static_cast<unsigned>(n), TILE_THR, 0, st>>>(
        tiles, mats, ws, 0, 0, c);
    return hipGetLastError();
}

hipError_t launch_ortho_apply(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                              int32_t src, bool first, bool last, OrthoCoef c, hipStream_t st) {
    if (n == 0) return hipSuccess;
    if (last)
        ortho_product_kernel<kLast, TILE_ARGS><<<static_cast<unsigned>(n), TILE_THR, 0, st>>>(
            tiles, mats, ws, src, first, c);
    else
        ortho_product_kernel<kApply, TILE_ARGS><<<static_cast<unsigned>(n), TILE_THR, 0, st>>>(
            tiles, mats, ws, src, first, c);
    return hipGetLastError();
}

}  // namespace fsdp
