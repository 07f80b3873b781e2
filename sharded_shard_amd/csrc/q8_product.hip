// Products of 8-bit matrices with a power of two for each block of 128, on the
// matrix cores: out = op(a) op(b), 32-bit sums, one rounding to bf16.
//
// One instruction takes 16 x 16 results and 128 of the sum, which is one block:
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies its 32-element stretches by the
// powers of two of both operands, so the scales cost the sum nothing.  Rows i
// of the results (M, from `a`) are the instruction's columns and columns j (N,
// from `b`) its rows: a lane then has neighbouring j of one i.
//
// Inside the instruction eight neighbouring products at a time are aligned to
// the largest of them and what lies 2^-14 below its power of two is dropped
// (measured); the eights and the accumulator add in fp32.  A sum is so within
// 7 2^-13 of its largest products, 1.5e-5 of the result for normal data and
// below the 2^-9 of the rounding to bf16 that follows.
#include "q8.hpp"

#include "device.hpp"

namespace fsdp {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) uint32_t lds_u32;
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
typedef __attribute__((address_space(3))) i32x4 lds_i32x4;

// elements of the sum a step: one block's side
constexpr int kBK = 128;

// How the codes of an operand lie: rows of the sum's elements, or the sum's
// elements one row after the other.
struct Operand {
    const char *codes;
    const uint8_t *scales;
    int64_t ld, pitch;
    int32_t n;              // rows of results (a) or columns (b)
    int32_t blocks;
};

// ---------------------------------------------------------------------------
// LDS images of a step
// ---------------------------------------------------------------------------

// Rows of 128 bytes: a row's 16-byte chunk sits at its index xor this.  The 16
// rows of one operand read hit all 64 banks.
__device__ __forceinline__ int swz_row(int row) { return (row >> 1) & 7; }

// The sum's elements as rows of W bytes: what a row's chunks are xored with, so
// that the eight rows of a transposing read, and eight rows 16 further, which
// the same LDS cycle reads, hit all banks.
template <int W>
__device__ __forceinline__ int swz_col(int k) {
    if constexpr (W == 256) return (k & 7) | (k >> 1 & 8);
    else if constexpr (W == 128) return (k >> 1 & 3) | (k >> 2 & 4);
    else return (k >> 2 & 1) | (k >> 3 & 2);
}

// In a 64-row stretch of b's rows, row 16 t + j of the image is row 4 j + t: the
// results of a lane, which come from rows 4 g .. + 4 of every 16, are then 16
// neighbouring columns, and one dword has the scales of its four rows.
__device__ __forceinline__ int spread(int r) {
    return (r & ~63) | (r & 15) << 2 | (r >> 4 & 3);
}

constexpr uint32_t kPastAll = 0x7FFFFFF0u;

// This wave's share of an operand's image, W rows (or columns) of results and one
// step of the sum: loads of 1 KB each straight into LDS, every WAVES-th one.  Rows,
// columns and elements past the matrix become zeros, whole 16 bytes at a time.
template <bool kCol, int W, bool kSpread, int WAVES>
struct Filler {
    static constexpr int kLoads = W / 8 / WAVES;
    static_assert(W / 8 % WAVES == 0 && WAVES % 2 == 0, "whole loads; chunks the same for all");
    const char *base;
    uint32_t voff, ld, nbytes;      // of load 0 and element 0; rows past the matrix lie past nbytes
    int K, chunk;

    __device__ __forceinline__ Filler(const Operand &O, int i0, int K_, int wave, int lane)
        : ld(static_cast<uint32_t>(O.ld)), K(K_) {
        const int left = O.n - i0;
        if constexpr (!kCol) {
            const int rho = 8 * wave + (lane >> 3);
            chunk = 16 * ((lane & 7) ^ swz_row(rho));
            voff = static_cast<uint32_t>(kSpread ? spread(rho) : rho) * ld + chunk;
            base = O.codes + static_cast<int64_t>(i0) * O.ld;
            nbytes = static_cast<uint32_t>((left < W ? left : W) - 1) * ld + ((K + 15) & ~15);
        } else {
            constexpr int kChunks = W / 16, kRows = 1024 / W;
            const int k = wave * kRows + lane / kChunks, c = 16 * (lane % kChunks ^ swz_col<W>(k));
            chunk = 0;
            voff = c < left ? static_cast<uint32_t>(k) * ld + c : kPastAll;
            base = O.codes + i0;
            nbytes = static_cast<uint32_t>((left + 15) & ~15);
        }
    }
    // load t of step s
    __device__ __forceinline__ void load(lds_char *image, int s, int t, int wave) const {
        const int k0 = s * kBK;
        const char *b = base;
        uint32_t n = nbytes, o;
        if constexpr (!kCol) {
            const int rows = kSpread ? spread(t * 8 * WAVES) : t * 8 * WAVES;
            o = k0 + chunk < K ? voff + (static_cast<uint32_t>(rows) * ld + k0) : kPastAll;
        } else {
            b += static_cast<int64_t>(k0) * ld;
            n += static_cast<uint32_t>((K - k0 < kBK ? K - k0 : kBK) - 1) * ld;
            o = voff + static_cast<uint32_t>(t * WAVES * (1024 / W)) * ld;
        }
        const __amdgpu_buffer_rsrc_t r =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(b), 0, n, 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            r, (lds_void *)(image + (t * WAVES + wave) * 1024), 16, o, 0, 0, 0);
    }
};

// 16 rows (results) and 128 elements of the sum: lane l has row l & 15 and the
// 16-byte chunks l >> 4 and 4 + (l >> 4) of it, whichever form it comes from.
union Frag {
    i32x8 v;
    i32x4 h[2];
    i32x2 q[4];
};

__device__ __forceinline__ i32x8 read_rows(const lds_char *t, int row0, int lane) {
    const int row = row0 + (lane & 15), g = lane >> 4;
    const lds_char *p = t + row * 128;
    Frag f;
    f.h[0] = *(const lds_i32x4 *)(p + (g ^ swz_row(row)) * 16);
    f.h[1] = *(const lds_i32x4 *)(p + ((4 + g) ^ swz_row(row)) * 16);
    return f.v;
}

// Eight rows of 16 bytes, turned over: lane l of 16 gives the address of 8
// bytes of row l >> 1 and gets byte l & 7 of those that the lanes 2 i + (l >> 3)
// name.  (restrict: no wait for loads to LDS that are under way.)
__device__ __forceinline__ i32x2 read_tr(lds_char *__restrict__ t) {
    return __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2 *)t);
}

template <int W>
__device__ __forceinline__ i32x8 read_cols(lds_char *t, int col0, int lane) {
    const int g = lane >> 4, l = lane & 15;
    Frag f;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const int k = (h >> 1) * 64 + 16 * g + (h & 1) * 8 + (l >> 1);
        f.q[h] = read_tr(t + k * W + (((col0 >> 4) ^ swz_col<W>(k)) * 16) + (l & 1) * 8);
    }
    return f.v;
}

// ---------------------------------------------------------------------------
// scales
// ---------------------------------------------------------------------------

// Of 128 results' scales in LDS, byte x of the pair is that of this lane's row of
// the x-th 16.
__device__ __forceinline__ i32x2 spread_scales(lds_char *t, int lane) {
    return read_tr(t + (lane & 15) * 8);
}

// ---------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------

struct Out {
    uint16_t *p;
    float *sums;            // fp32 [split, M, N] in place of p
    const float *div_a, *div_b;
    int64_t ld;
    int32_t split;
};

__device__ __forceinline__ float factor(const Out &o) {
    return 1.0f / (o.div_a ? *o.div_a : 1.0f) / (o.div_b ? *o.div_b : 1.0f);
}

template <int N>
struct Int {
    static constexpr int value = N;
};
// f(Int<0>) ... f(Int<N - 1>)
template <int N, int I = 0, typename F>
__device__ __forceinline__ void for_each(F &&f) {
    if constexpr (I < N) {
        f(Int<I>{});
        for_each<N, I + 1>(f);
    }
}

// The tile of this block.  Blocks go round-robin over the 8 XCDs; each XCD takes a
// stretch of an order in which eight rows of tiles are worked off column by column,
// so that what its blocks read at a time fits its L2.
__device__ __forceinline__ void tile_of(int tiles_m, int tiles_n, int &ti, int &tj) {
    constexpr int kRows = 8;
    const int n = tiles_m * tiles_n, b = blockIdx.x, xcd = b & 7, per = n >> 3, rem = n & 7;
    const int t = xcd * per + (xcd < rem ? xcd : rem) + (b >> 3);
    const int group = t / (kRows * tiles_n), first = group * kRows;
    const int rows = tiles_m - first < kRows ? tiles_m - first : kRows;
    const int at = t - first * tiles_n;
    ti = first + at % rows;
    tj = at / rows;
}

// n neighbouring results of row i from column j.
template <int n, typename F>
__device__ __forceinline__ void store(const Out &o, float f, int part, int i, int j, int M, int N, F &&get) {
    if (o.sums != nullptr) {
        float *p = o.sums + (static_cast<int64_t>(part) * M + i) * N + j;
        const bool vec = j + n <= N && (N & 3) == 0;
#pragma unroll
        for (int e = 0; e < n; e += 4) {
            if (vec) {
                *reinterpret_cast<f32x4 *>(p + e) = f32x4{get(e), get(e + 1), get(e + 2), get(e + 3)};
            } else {
#pragma unroll
                for (int t = e; t < e + 4; ++t)
                    if (j + t < N) p[t] = get(t);
            }
        }
        return;
    }
    uint16_t *p = o.p + static_cast<int64_t>(i) * o.ld + j;
    uint32_t w[n / 2];
#pragma unroll
    for (int e = 0; e < n; e += 2) w[e / 2] = pack2(get(e) * f, get(e + 1) * f);
    constexpr int kVec = n == 4 ? 4 : 8;        // results a store
    if (j + n <= N && (lo32(o.p) & (2 * kVec - 1)) == 0 && (o.ld & (kVec - 1)) == 0) {
#pragma unroll
        for (int e = 0; e < n; e += kVec) {
            if constexpr (kVec == 4) *reinterpret_cast<u32x2 *>(p + e) = u32x2{w[0], w[1]};
            else
                *reinterpret_cast<u32x4 *>(p + e) =
                    u32x4{w[e / 2], w[e / 2 + 1], w[e / 2 + 2], w[e / 2 + 3]};
        }
    } else {
#pragma unroll
        for (int e = 0; e < n; ++e)
            if (j + e < N) p[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
    }
}

// The scales of an operand's W results, four a lane and one dword a step: as they lie,
// or a 128 x 128 block's one byte four times over.
template <int W>
struct ScaleLoader {
    const uint8_t *base;
    int64_t step;
    uint32_t voff, select, add, bits;
    __device__ __forceinline__ ScaleLoader(const Operand &O, bool col, int i0, int lane) {
        int i = 4 * (lane % (W / 4));
        i = i0 + i < O.n ? i : (O.n - 1 - i0) & ~3;
        base = O.scales, step = 0, voff = 0, select = 0x0C0C0C0Cu, add = 0u, bits = 0u;
        if (O.blocks == FSDP_Q8_TENSOR) {       // 2^0, whatever lies there
            base = reinterpret_cast<const uint8_t *>(O.codes);
            bits = 0x7F7F7F7Fu;
        } else if (O.blocks == FSDP_Q8_TILES) {
            base += col ? i0 >> 7 : static_cast<int64_t>(i0 >> 7) * O.pitch;
            voff = static_cast<uint32_t>(i >> 7) * (col ? 1u : static_cast<uint32_t>(O.pitch));
            step = col ? O.pitch : 1, select = 0u, add = 0x01010101u;
        } else {
            base += i0;
            voff = i, step = O.pitch, select = 0x03020100u;
        }
    }
};

template <int N>
__device__ __forceinline__ void border() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// One BM x BN tile a block, WM x WN waves of FM x 4 results of 16 x 16 each.  Two
// images in LDS.  A step's products are made in two halves of the wave's rows i.
// During the first half the second half's rows are read, after which the step's
// image is free; at the border in the middle every wave has them in registers
// and the next step's image has landed; during the second half the next step's
// first rows and, as their last products are made, its columns are read, and the
// step after it starts on its way into the freed image.
template <int BM, int BN, int WM, int WN, bool kColA, bool kColB, int FMTA>
__global__ __launch_bounds__(64 * WM *WN, 2) void q8_product_kernel(Operand A, Operand B, Out out,
                                                                    int K) {
    constexpr int WAVES = WM * WN, WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
    constexpr int HM = FM / 2;
    constexpr int kStage = (BM + BN) * kBK;
    // scales in LDS: 128 bytes may be read past a wave's own
    constexpr int kScalesB = BM + 128, kScales = kScalesB + BN + 128;
    static_assert(FN == 4 && FM % 2 == 0 && FM <= 8, "");
    __shared__ __attribute__((aligned(1024))) char smem[2 * kStage + 2 * kScales];
    lds_char *lds = (lds_char *)smem;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN, g = lane >> 4;
    const int tiles_m = (A.n + BM - 1) / BM, tiles_n = (B.n + BN - 1) / BN;
    int ti, tj;
    tile_of(tiles_m, tiles_n, ti, tj);
    const int i0 = ti * BM, j0 = tj * BN, part = blockIdx.y;
    const int all = (K + kBK - 1) / kBK;
    // at most 2^15 steps, in far fewer stretches than 2^16
    const int from = static_cast<int>(static_cast<uint32_t>(all * part) / static_cast<uint32_t>(out.split));
    const int to = static_cast<int>(static_cast<uint32_t>(all * (part + 1)) / static_cast<uint32_t>(out.split));

    f32x4 acc[FM][FN];
#pragma unroll
    for (int x = 0; x < FM; ++x)
#pragma unroll
        for (int y = 0; y < FN; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    if (from < to) {
        const Filler<kColA, BM, false, WAVES> fa(A, i0, K, wave, lane);
        const Filler<kColB, BN, !kColB, WAVES> fb(B, j0, K, wave, lane);
        constexpr int kLA = decltype(fa)::kLoads, kLB = decltype(fb)::kLoads;
        // even waves put a's scales into LDS, odd ones b's, all of them over and over:
        // no branch
        const bool of_a = (wave & 1) == 0;
        const ScaleLoader<BM> la(A, kColA, i0, lane);
        const ScaleLoader<BN> lb(B, kColB, j0, lane);
        const uint8_t *sbase = of_a ? la.base : lb.base;
        const int64_t sstep = of_a ? la.step : lb.step;
        const uint32_t svoff = of_a ? la.voff : lb.voff, sselect = of_a ? la.select : lb.select,
                       sadd = of_a ? la.add : lb.add, sbits = of_a ? la.bits : lb.bits;
        const int sat = 2 * kStage + 4 * (of_a ? lane % (BM / 4) : kScalesB / 4 + lane % (BN / 4));
        uint32_t sw, ssel;
        auto load_scales = [&](int s) {
            const uint8_t *p = sbase + s * sstep + svoff;
            ssel = sselect + (lo32(p) & 3u) * sadd;
            sw = *reinterpret_cast<const uint32_t *>(p - (lo32(p) & 3u));
        };
        auto put_scales = [&](int s) {
            *(lds_u32 *)(lds + sat + (s & 1) * kScales) = __builtin_amdgcn_perm(sw, sw, ssel) | sbits;
        };
        auto image = [&](int s) { return lds + (s & 1) * kStage; };
        auto read_p = [&](int s, int x) {
            lds_char *t = image(s);
            if constexpr (kColA) return read_cols<BM>(t, wm * WTM + 16 * x, lane);
            else return read_rows(t, wm * WTM + 16 * x, lane);
        };
        auto read_q = [&](int s, int y) {
            lds_char *t = image(s) + BM * kBK;
            if constexpr (kColB) return read_cols<BN>(t, wn * WTN + 16 * y, lane);
            else return read_rows(t, wn * WTN + 16 * y, lane);
        };
        auto read_sa = [&](int s) {
            return spread_scales(lds + 2 * kStage + (s & 1) * kScales + wm * WTM, lane);
        };
        auto read_sb = [&](int s) {
            lds_char *t = lds + 2 * kStage + (s & 1) * kScales + kScalesB + wn * WTN;
            if constexpr (kColB) return spread_scales(t, lane).x;
            else return static_cast<int>(*(const lds_u32 *)(t + 4 * (lane & 15)));
        };
        // what follows the sum's last element in its 16 bytes is no part of it
        auto cut_tail = [&](int s) {
            if ((kColA && kColB) || s != all - 1 || (K & 15) == 0) return;
            const int c = (K & 127) >> 4, keep = K & 15;
            constexpr int kRowsA = kColA ? 0 : BM, kRowsB = kColB ? 0 : BN;
            for (int r = tid; r < kRowsA + kRowsB; r += 64 * WAVES) {
                const bool of_a = r < kRowsA;
                const int row = of_a ? r : r - kRowsA;
                lds_char *p = image(s) + (of_a ? 0 : BM * kBK) + row * 128 + (c ^ swz_row(row)) * 16;
                for (int b = keep; b < 16; ++b) p[b] = 0;
            }
            border<0>();
        };

        load_scales(from);
#pragma unroll
        for (int t = 0; t < kLA; ++t) fa.load(image(from), from, t, wave);
#pragma unroll
        for (int t = 0; t < kLB; ++t) fb.load(image(from) + BM * kBK, from, t, wave);
        put_scales(from);
        border<0>();
        cut_tail(from);
        i32x8 p[FM], q[FN];
        i32x2 sa = read_sa(from);
        int sb = read_sb(from);
#pragma unroll
        for (int x = 0; x < HM; ++x) p[x] = read_p(from, x);
#pragma unroll
        for (int y = 0; y < FN; ++y) q[y] = read_q(from, y);
        if (from + 1 < to) {
            load_scales(from + 1);
#pragma unroll
            for (int t = 0; t < kLA; ++t) fa.load(image(from + 1), from + 1, t, wave);
#pragma unroll
            for (int t = 0; t < kLB; ++t)
                fb.load(image(from + 1) + BM * kBK, from + 1, t, wave);
        }

        auto mma = [&](auto xc, auto yc) {
            constexpr int x = decltype(xc)::value, y = decltype(yc)::value;
            acc[x][y] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                q[y], p[x], acc[x][y], 0, FMTA, y, sb, x & 3, x < 4 ? sa.x : sa.y);
        };
        // kMore: steps that follow, 2 for two and more
        auto step = [&](int s, auto more) {
            constexpr int kMore = decltype(more)::value;
            // columns y outermost: the first products need the first columns alone
            for_each<HM * FN>([&](auto nc) {
                constexpr int n = decltype(nc)::value, y = n / HM, x = n % HM;
                mma(Int<x>{}, Int<y>{});
                // the second half's rows, one operand at a time, in the first products' time
                if constexpr (n < HM) p[HM + n] = read_p(s, HM + n);
                if constexpr (n == HM && kMore > 0) put_scales(s + 1);
                __builtin_amdgcn_sched_barrier(0);
            });
            i32x2 sa2 = sa;
            int sb2 = sb;
            if constexpr (kMore > 0) {
                border<0>();
                if constexpr (kMore == 1) cut_tail(s + 1);
                sa2 = read_sa(s + 1);
                sb2 = read_sb(s + 1);
                if constexpr (kMore > 1) load_scales(s + 2);
            }
            for_each<HM * FN>([&](auto nc) {
                constexpr int n = decltype(nc)::value, y = n / HM, x = n % HM;
                mma(Int<HM + x>{}, Int<y>{});
                if constexpr (kMore > 0) {
                    if constexpr (n < HM) p[n] = read_p(s + 1, n);
                    if constexpr (x == HM - 1) q[y] = read_q(s + 1, y);
                }
                if constexpr (kMore > 1) {
                    // the loads, spread over the half
                    constexpr int kL = kLA + kLB, lo = n * kL / (HM * FN),
                                  hi = (n + 1) * kL / (HM * FN);
                    for_each<hi - lo>([&](auto tc) {
                        constexpr int t = lo + decltype(tc)::value;
                        if constexpr (t < kLA) fa.load(image(s + 2), s + 2, t, wave);
                        else fb.load(image(s + 2) + BM * kBK, s + 2, t - kLA, wave);
                    });
                }
                __builtin_amdgcn_sched_barrier(0);
            });
            sa = sa2;
            sb = sb2;
        };
        int s = from;
        for (; s + 2 < to; ++s) step(s, Int<2>{});
        if (s + 1 < to) {
            step(s, Int<1>{});
            ++s;
        }
        step(s, Int<0>{});
    }

    // Row i of the results; this lane's columns: 16 neighbouring ones of every 64, or
    // four of every 16.
    const float f = factor(out);
    for_each<FM>([&](auto xc) {
        constexpr int x = decltype(xc)::value;
        const int i = i0 + wm * WTM + 16 * x + (lane & 15);
        if (i < A.n) {
            if constexpr (kColB) {
                for_each<FN>([&](auto yc) {
                    constexpr int y = decltype(yc)::value;
                    store<4>(out, f, part, i, j0 + wn * WTN + 16 * y + 4 * g, A.n, B.n,
                             [&](int e) { return acc[x][y][e]; });
                });
            } else {
                store<16>(out, f, part, i, j0 + wn * WTN + 16 * g, A.n, B.n,
                          [&](int e) { return acc[x][e & 3][e >> 2]; });
            }
        }
    });
}

// The stretches' sums in order.
__global__ __launch_bounds__(kBlock) void q8_join_kernel(Out out, int M, int N) {
    const int64_t n = static_cast<int64_t>(M) * N;
    const float f = factor(out);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kBlock) {
        float s = out.sums[i];
        for (int k = 1; k < out.split; ++k) s += out.sums[k * n + i];
        const int64_t row = i / N;
        out.p[row * out.ld + (i - row * N)] = static_cast<uint16_t>(bf16_rne(s * f));
    }
}

// Rows of any alignment to rows of whole 16 bytes.
__global__ __launch_bounds__(kBlock) void q8_align_kernel(const uint8_t *from, int64_t ld, int rows,
                                                          int cols, uint8_t *to, int64_t ldo) {
    const int64_t per = ldo >> 4, n = per * rows;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kBlock) {
        const int64_t r = i / per, c = (i - r * per) * 16;
        const uint8_t *p = from + r * ld + c;
        u32x4 w{0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (c + e < cols) w[e >> 2] |= static_cast<uint32_t>(p[e]) << (8 * (e & 3));
        reinterpret_cast<u32x4 *>(to)[i] = w;
    }
}

unsigned blocks_for(int64_t n) {
    const int64_t b = (n + kBlock - 1) / kBlock;
    return static_cast<unsigned>(b < 8192 ? b : 8192);
}

template <int BM, int BN, int WM, int WN>
void launch(const Operand &A, bool ta, const Operand &B, bool tb, int format, const Out &out, int K,
            hipStream_t st) {
    const dim3 grid((A.n + BM - 1) / BM * ((B.n + BN - 1) / BN), out.split);
    const bool e4 = format == FSDP_Q8_E4M3;
    void (*kernel)(Operand, Operand, Out, int) = nullptr;
    if (!ta && tb)
        kernel = e4 ? q8_product_kernel<BM, BN, WM, WN, false, false, 0>
                    : q8_product_kernel<BM, BN, WM, WN, false, false, 1>;
    else if (!ta)
        kernel = e4 ? q8_product_kernel<BM, BN, WM, WN, false, true, 0>
                    : q8_product_kernel<BM, BN, WM, WN, false, true, 1>;
    else
        kernel = e4 ? q8_product_kernel<BM, BN, WM, WN, true, true, 0>
                    : q8_product_kernel<BM, BN, WM, WN, true, true, 1>;
    kernel<<<grid, 64 * WM * WN, 0, st>>>(A, B, out, K);
}

int64_t round16(int64_t x) { return (x + 15) & ~int64_t{15}; }
int64_t round256(int64_t x) { return (x + 255) & ~int64_t{255}; }

bool aligned(const Q8Mat &m) {
    return (reinterpret_cast<uintptr_t>(m.codes) & 15u) == 0 && (m.ld & 15) == 0;
}

}  // namespace

Q8Cut q8_cut(const Q8Mat &a, bool ta, const Q8Mat &b, bool tb) {
    const int M = ta ? a.cols : a.rows, N = tb ? b.rows : b.cols;
    Q8Cut c{};
    c.tile = M <= 64 || N <= 64 ? 2 : M <= 128 || N <= 128 ? 1 : 0;
    c.split = 1;
    c.bytes_a = aligned(a) ? 0 : round256(round16(a.cols) * a.rows);
    c.bytes_b = aligned(b) ? 0 : round256(round16(b.cols) * b.rows);
    c.bytes_sums = c.split == 1 ? 0 : int64_t{4} * M * N * c.split;
    return c;
}

hipError_t launch_q8_product(const Q8Mat &a, bool ta, const Q8Mat &b, bool tb, uint16_t *p,
                             int64_t ldo, const Q8Cut &cut, void *ws, hipStream_t st) {
    const int M = ta ? a.cols : a.rows, N = tb ? b.rows : b.cols, K = ta ? a.rows : a.cols;
    if (M == 0 || N == 0) return hipSuccess;
    char *at = static_cast<char *>(ws);
    auto operand = [&](const Q8Mat &m, int64_t bytes, int n) {
        Operand o{reinterpret_cast<const char *>(m.codes), m.scales, m.ld, m.pitch, n, m.blocks};
        if (bytes > 0 && K > 0) {
            o.ld = round16(m.cols);
            q8_align_kernel<<<blocks_for(o.ld / 16 * m.rows), kBlock, 0, st>>>(
                m.codes, m.ld, m.rows, m.cols, reinterpret_cast<uint8_t *>(at), o.ld);
            o.codes = at;
        }
        at += bytes;
        return o;
    };
    const Operand A = operand(a, cut.bytes_a, M), B = operand(b, cut.bytes_b, N);
    Out out{p, cut.split > 1 ? reinterpret_cast<float *>(at) : nullptr, a.divisor, b.divisor, ldo,
            cut.split};
    if (cut.tile == 0) launch<256, 256, 2, 4>(A, ta, B, tb, a.format, out, K, st);
    else if (cut.tile == 1) launch<128, 128, 2, 2>(A, ta, B, tb, a.format, out, K, st);
    else launch<64, 64, 2, 1>(A, ta, B, tb, a.format, out, K, st);
    if (cut.split > 1)
        q8_join_kernel<<<blocks_for(static_cast<int64_t>(M) * N), kBlock, 0, st>>>(out, M, N);
    return hipGetLastError();
}

}  // namespace fsdp
