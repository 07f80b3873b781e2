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
// Layout.  Only X^T is stored, [np][mp].  X = a X + B X is then a product of
// rows with rows (rows of B, rows of X^T), and A sums over rows of X^T, whose
// tiles the transposing LDS read turns into operands.
#include "ortho.hpp"

#include "device.hpp"

namespace fsdp {

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) f16x8 lds_f16x8;

// log2 of the scale of A and B
constexpr int kLogA = 11;
// log2 of the scale of X where the norm is not lost in eps
constexpr int kLogX = 12;

__device__ __forceinline__ char *at(void *ws, int64_t off) { return static_cast<char *>(ws) + off; }

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
        const int64_t o = static_cast<int64_t>(tl.tj * 64 + y) * M.mp + tl.ti * 64 + tx;
        hi[o] = h;
        lo[o] = static_cast<_Float16>(x - static_cast<float>(h));
    }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

enum { kGram = 0, kPoly = 1, kApply = 2, kLast = 3 };

constexpr int kBK = 64;

// A 32 x 32 block's rows come back from the matrix core as four runs of four a
// lane; with operand row rho holding tile row pi(rho) a lane's values are two
// runs of eight neighbouring rows instead: 16-byte stores.
//   rho = 8 (2c + d) + 4 h + e  ->  16 c + 8 h + 4 d + e
__device__ __forceinline__ int perm_row(int rho) {
    const int e = rho & 3, h = (rho >> 2) & 1, d = (rho >> 3) & 1, c = rho >> 4;
    return 16 * c + 8 * h + 4 * d + e;
}

// Tiles of rows with 64 halves (128 bytes, eight 16-byte chunks): the chunk
// sits at its index xor this, so that the eight lanes of one LDS cycle, which
// read eight rows at the same index, hit different banks.
__device__ __forceinline__ int swz_row(int row) { return (row & 3) | ((row >> 1) & 4); }

// Fills `rows` rows of an LDS tile from a row-major matrix (ld bytes a row,
// rows past `avail` bytes read zeros): each wave's load writes 1 KB, 8 rows.
template <int ROWS, int WAVES>
__device__ __forceinline__ void fill_rows(lds_char *dst, const char *src, uint32_t ld,
                                          uint32_t avail, uint32_t kbyte, int wave, int lane) {
    static_assert(ROWS % (8 * WAVES) == 0, "whole loads per wave");
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char *>(src), 0, avail, 0x00020000);
#pragma unroll
    for (int i = 0; i < ROWS / 8 / WAVES; ++i) {
        const int row8 = (i * WAVES + wave) * 8, row = row8 + (lane >> 3);
        const uint32_t voff = static_cast<uint32_t>(row) * ld +
                              static_cast<uint32_t>((lane & 7) ^ swz_row(row)) * 16u;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(dst + row8 * 128), 16, voff, kbyte,
                                                 0, 0);
    }
}

// Fills a tile of kBK rows of COLS halves (the sum runs over rows).  A
// 32-byte piece p of row k sits at p xor swz_col(k): a transposing read takes
// 32 bytes of each of 16 rows at the same p.
__device__ __forceinline__ int swz_col(int k) { return (k & 3) | ((k >> 1) & 4); }

template <int COLS, int WAVES>
__device__ __forceinline__ void fill_cols(lds_char *dst, const char *src, uint32_t ld,
                                          uint32_t avail, uint32_t kbyte, int wave, int lane) {
    constexpr int kPer = 1024 / (COLS * 2);       // rows per load
    constexpr int kLanes = 64 / kPer;             // lanes per row
    static_assert(kBK % (kPer * WAVES) == 0, "whole loads per wave");
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char *>(src), 0, avail, 0x00020000);
#pragma unroll
    for (int i = 0; i < kBK / kPer / WAVES; ++i) {
        const int k0 = (i * WAVES + wave) * kPer, k = k0 + lane / kLanes, c = lane % kLanes;
        const uint32_t voff = static_cast<uint32_t>(k) * ld +
                              static_cast<uint32_t>(((c >> 1) ^ swz_col(k)) * 32 + (c & 1) * 16);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(dst + k0 * COLS * 2), 16, voff,
                                                 kbyte, 0, 0);
    }
}

// Operand of 32 rows and 16 k: this lane's row and its 8 k.
__device__ __forceinline__ f16x8 read_rows(const lds_char *t, int row, int ks, int lane) {
    const int c = (ks * 2 + (lane >> 5)) ^ swz_row(row);
    return *(const lds_f16x8 *)(t + row * 128 + c * 16);
}

// The same from a tile with the sum over rows.  Lane l of a 16-lane group reads
// 4 neighbouring columns (8 bytes) of row k0 + (l >> 2); it gets column l of
// the 16 that lanes 0 to 3 read, of those 4 rows.  col: the first column that
// this lane reads.
template <int COLS>
__device__ __forceinline__ f16x8 read_cols(lds_char *t, int col, int ks, int lane) {
    const int k0 = ks * 16 + (lane >> 5) * 8 + ((lane >> 2) & 3);
    union {
        s16x4 s[2];
        f16x8 v;
    } u;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int k = k0 + 4 * j;
        u.s[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4 *)(t + k * COLS * 2 + (((col >> 4) ^ swz_col(k)) * 32) + (col & 15) * 2));
    }
    return u.v;
}

// Bytes of `rows` rows, as far as a buffer range reaches (a tile needs less).
__device__ __forceinline__ uint32_t bytes_from(int rows, uint32_t ld) {
    const int64_t b = static_cast<int64_t>(rows) * ld;
    return b > 0x7FFFFFFF ? 0x7FFFFFFFu : static_cast<uint32_t>(b);
}

template <int KIND, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM *WN) void ortho_product_kernel(
    const OrthoTile *__restrict__ tiles, const OrthoMat *__restrict__ mats, void *ws, int32_t src,
    int32_t first, OrthoCoef coef) {
    constexpr int WAVES = WM * WN, WTM = BM / WM, WTN = BN / WN, FM = WTM / 32, FN = WTN / 32;
    constexpr bool kSym = KIND == kGram || KIND == kPoly;
    constexpr int kStage = (BM + BN) * kBK * 2;
    __shared__ __attribute__((aligned(1024))) char smem[2 * kStage];
    lds_char *lds = (lds_char *)smem;

    const OrthoTile tl = tiles[blockIdx.x];
    const OrthoMat M = mats[tl.mat];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int i0 = tl.ti * BM, j0 = tl.tj * BN;

    // P gives the tile's rows i, Q its columns j
    const char *P, *Q;
    uint32_t ldk, availP, availQ, kstep;
    int K;
    if constexpr (KIND == kGram) {
        // rows of X^T are the sum: a stage is kBK of them, columns i0.. and j0..
        const char *T = at(ws, src ? M.t[1] : M.t[0]);
        P = T + i0 * 2;
        Q = T + j0 * 2;
        ldk = static_cast<uint32_t>(M.mp) * 2;
        availP = availQ = kBK * ldk;   // at most: the last columns' rows end before it
        K = M.np;
        kstep = 0;
    } else {
        const char *A = at(ws, KIND == kPoly ? M.a : M.b);
        ldk = static_cast<uint32_t>(M.mp) * 2;
        P = A + static_cast<int64_t>(i0) * ldk;
        Q = KIND == kPoly ? A + static_cast<int64_t>(j0) * ldk
                          : at(ws, src ? M.t[1] : M.t[0]) + static_cast<int64_t>(j0) * ldk;
        availP = bytes_from(M.mp - i0, ldk);
        availQ = bytes_from((KIND == kPoly ? M.mp : M.np) - j0, ldk);
        K = M.mp;
        kstep = kBK * 2;
    }

    f32x16 acc[FM][FN];
#pragma unroll
    for (int x = 0; x < FM; ++x)
#pragma unroll
        for (int y = 0; y < FN; ++y)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[x][y][e] = 0.0f;

    auto fill = [&](int s, int buf) {
        lds_char *b = lds + buf * kStage;
        if constexpr (KIND == kGram) {
            const int64_t o = static_cast<int64_t>(s) * kBK * ldk;
            fill_cols<BM, WAVES>(b, P + o, ldk, availP, 0, wave, lane);
            fill_cols<BN, WAVES>(b + BM * kBK * 2, Q + o, ldk, availQ, 0, wave, lane);
        } else {
            fill_rows<BM, WAVES>(b, P, ldk, availP, s * kstep, wave, lane);
            fill_rows<BN, WAVES>(b + BM * kBK * 2, Q, ldk, availQ, s * kstep, wave, lane);
        }
    };

    const int steps = K / kBK;
    // both operands take their rows through the same permutation
    const int prow = perm_row(lane & 31);
    const int pcol = perm_row((lane & 16) | ((lane & 3) << 2));
    fill(0, 0);
    for (int s = 0; s < steps; ++s) {
        // the wave's own loads of stage s have landed; past the barrier so have
        // the others', and nobody reads the other buffer any more
        __builtin_amdgcn_s_waitcnt(0x0F70);       // vmcnt(0)
        __syncthreads();
        if (s + 1 < steps) fill(s + 1, (s + 1) & 1);
        lds_char *b = lds + (s & 1) * kStage;
        lds_char *bp = b, *bq = b + BM * kBK * 2;
#pragma unroll
        for (int ks = 0; ks < kBK / 16; ++ks) {
            f16x8 p[FM], q[FN];
#pragma unroll
            for (int x = 0; x < FM; ++x) {
                const int base = wm * WTM + x * 32;
                if constexpr (KIND == kGram) p[x] = read_cols<BM>(bp, base + pcol, ks, lane);
                else p[x] = read_rows(bp, base + prow, ks, lane);
            }
#pragma unroll
            for (int y = 0; y < FN; ++y) {
                const int base = wn * WTN + y * 32;
                if constexpr (KIND == kGram) q[y] = read_cols<BN>(bq, base + pcol, ks, lane);
                else q[y] = read_rows(bq, base + prow, ks, lane);
            }
#pragma unroll
            for (int x = 0; x < FM; ++x)
#pragma unroll
                for (int y = 0; y < FN; ++y)
                    acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(p[x], q[y], acc[x][y], 0, 0,
                                                                       0);
        }
    }

    // Epilogue.  Of block (x, y) this lane has column j and, for c = 0, 1, the
    // rows 16 c + 8 h .. + 8 in acc[8 c .. 8 c + 8).
    const OrthoScal sc = *reinterpret_cast<const OrthoScal *>(at(ws, M.scal));
    const int h = lane >> 5;
    if constexpr (kSym) {
        _Float16 *C = reinterpret_cast<_Float16 *>(at(ws, KIND == kGram ? M.a : M.b));
        const _Float16 *A = reinterpret_cast<const _Float16 *>(at(ws, M.a));
        const float phi = first ? sc.phi0 : sc.phi;
        const float alpha = KIND == kGram ? ldexpf(phi * phi, kLogA) : ldexpf(coef.c, -kLogA);
#pragma unroll
        for (int x = 0; x < FM; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int i = i0 + wm * WTM + x * 32 + 16 * c + 8 * h;
                    const int j = j0 + wn * WTN + y * 32 + prow;
                    if (i >= M.mp || j >= M.mp) continue;
                    f16x8 v;
                    f16x8 old;
                    if constexpr (KIND == kPoly)
                        old = *reinterpret_cast<const f16x8 *>(A + static_cast<int64_t>(j) * M.mp + i);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float t = alpha * acc[x][y][8 * c + e];
                        if constexpr (KIND == kPoly) t = coef.b * static_cast<float>(old[e]) + t;
                        v[e] = static_cast<_Float16>(t);
                    }
                    // (i, j) and (j, i) are the same value; a diagonal tile has
                    // both among its own, which must not differ: the lower wins
                    if (tl.ti != tl.tj) {
                        *reinterpret_cast<f16x8 *>(C + static_cast<int64_t>(j) * M.mp + i) = v;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            C[static_cast<int64_t>(i + e) * M.mp + j] = v[e];
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (i + e >= j) {
                                C[static_cast<int64_t>(i + e) * M.mp + j] = v[e];
                                C[static_cast<int64_t>(j) * M.mp + i + e] = v[e];
                            }
                    }
                }
    } else {
        const _Float16 *T = reinterpret_cast<const _Float16 *>(at(ws, src ? M.t[1] : M.t[0]));
        _Float16 *T2 = reinterpret_cast<_Float16 *>(at(ws, src ? M.t[0] : M.t[1]));
        _Float16 *L = reinterpret_cast<_Float16 *>(at(ws, M.lo));
        const float rho = first ? sc.rho : 1.0f;
        const float ca = coef.a * rho, cb = ldexpf(rho, -kLogA);
#pragma unroll
        for (int x = 0; x < FM; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int i = i0 + wm * WTM + x * 32 + 16 * c + 8 * h;
                    const int j = j0 + wn * WTN + y * 32 + prow;
                    if (i >= M.mp || j >= M.np) continue;
                    const int64_t o = static_cast<int64_t>(j) * M.mp + i;
                    const f16x8 hi = *reinterpret_cast<const f16x8 *>(T + o);
                    const f16x8 lo = *reinterpret_cast<const f16x8 *>(L + o);
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = ca * (static_cast<float>(hi[e]) + static_cast<float>(lo[e])) +
                               cb * acc[x][y][8 * c + e];
                    if constexpr (KIND == kApply) {
                        f16x8 vh, vl;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            vh[e] = static_cast<_Float16>(v[e]);
                            vl[e] = static_cast<_Float16>(v[e] - static_cast<float>(vh[e]));
                        }
                        *reinterpret_cast<f16x8 *>(T2 + o) = vh;
                        *reinterpret_cast<f16x8 *>(L + o) = vl;
                    } else {
                        if (j >= M.n) continue;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            if (i + e >= M.m) continue;
                            const uint16_t w = static_cast<uint16_t>(bf16_rne(v[e] * sc.phi));
                            if (M.wide) M.out[static_cast<int64_t>(i + e) * M.cols + j] = w;
                            else M.out[static_cast<int64_t>(j) * M.cols + i + e] = w;
                        }
                    }
                }
    }
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

hipError_t launch_ortho_gram(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             int32_t src, bool first, hipStream_t st) {
    if (n == 0) return hipSuccess;
    ortho_product_kernel<kGram, 128, 128, 2, 2><<<static_cast<unsigned>(n), 256, 0, st>>>(
        tiles, mats, ws, src, first, OrthoCoef{});
    return hipGetLastError();
}

hipError_t launch_ortho_poly(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                             OrthoCoef c, hipStream_t st) {
    if (n == 0) return hipSuccess;
    ortho_product_kernel<kPoly, 128, 128, 2, 2><<<static_cast<unsigned>(n), 256, 0, st>>>(
        tiles, mats, ws, 0, 0, c);
    return hipGetLastError();
}

hipError_t launch_ortho_apply(const OrthoTile *tiles, int64_t n, const OrthoMat *mats, void *ws,
                              int32_t src, bool first, bool last, OrthoCoef c, hipStream_t st) {
    if (n == 0) return hipSuccess;
    if (last)
        ortho_product_kernel<kLast, 128, 128, 2, 2><<<static_cast<unsigned>(n), 256, 0, st>>>(
            tiles, mats, ws, src, first, c);
    else
        ortho_product_kernel<kApply, 128, 128, 2, 2><<<static_cast<unsigned>(n), 256, 0, st>>>(
            tiles, mats, ws, src, first, c);
    return hipGetLastError();
}

}  // namespace fsdp
