// Products of 8-bit matrices with a power of two for each block of 128, on the
// matrix cores: out = op(a) op(b), 32-bit sums, one rounding to bf16.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes 16 x 16 results and 128 of the sum, which
// is one block, and multiplies its 32-element stretches by the powers of two of both
// operands: the scales cost the sum nothing.  Rows i of the results (M, from `a`)
// are the instruction's columns and columns j (N, from `b`) its rows: a lane then
// has neighbouring j of one i.
//
// Inside the instruction eight neighbouring products at a time are aligned to
// the largest of them and keep their bits down to 2^-13 of its power of two
// (measured); the eights and the accumulator add in fp32.  An eight is so within
// 7 2^-13 of its largest product.  A sum is off by 1.5e-5 of its size on normal data
// and 4.5e-5 where one channel in a hundred is twenty times the others (root mean
// squares of fp32 sums of 8192), against up to 2^-8 in the rounding to bf16 that
// follows; where products cancel, by up to 2^-10 of the sum of their magnitudes.  That
// is the choice of 8-bit instructions: fp16 ones, exact here, run at half the rate.
#include "q8.hpp"

#include "device.hpp"
#include "q8_device.hpp"

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

// Rows of 128 bytes (whole cache lines: rows of 64 in twice as many steps took 474 us
// for 424 of a forward product): a row's 16-byte chunk sits at its index xor this,
// so that the 16 rows of one operand read hit all 64 banks.
__device__ __forceinline__ int swz_row(int row) { return (row >> 1) & 7; }

// The sum's elements as rows of W bytes: what a row's chunks are xored with, so
// that the eight rows of a transposing read, and eight rows 16 further, which
// the same LDS cycle reads, hit all banks.
template <int W>
__device__ __forceinline__ int swz_col(int k) {
    if constexpr (W == 256) return (k & 7) | (k >> 1 & 8);
    else if constexpr (W == 128) return (k >> 1 & 3) | (k >> 2 & 4);
    else if constexpr (W == 64) return (k >> 2 & 1) | (k >> 3 & 2);
    else return k >> 4 & 1;
}

// In a 64-row stretch of b's rows, row 16 t + 4 g + e of the image is row 32 (t >> 1) +
// 8 g + 4 (t & 1) + e: the results of a lane, which come from rows 4 g + e of every
// 16, are then twice eight neighbouring columns, and four lanes' next to each other.
__device__ __forceinline__ int spread(int r) {
    return (r & ~63) | (r & 32) | (r & 12) << 1 | (r & 16) >> 2 | (r & 3);
}
// The same turned over, for fours of rows.
__device__ __forceinline__ int spread_four(int d) {
    return (d & ~15) | (d & 8) | (d & 1) << 2 | (d & 6) >> 1;
}

constexpr uint32_t kPastAll = 0x7FFFFFF0u;

// Where the W rows (or columns) of results from i0 lie; past `size` bytes there are
// none.  No branch: one in a step would let products sink past its border.
template <bool kCol, int W>
struct Source {
    const char *base;
    uint32_t size;
    int left;
    __device__ __forceinline__ void aim(const Operand &O, int i0, int K) {
        left = O.n - i0 < 0 ? 0 : O.n - i0;
        base = O.codes + (kCol ? int64_t{i0} : i0 * O.ld);
        const int rows = left < W ? left : W;
        size = kCol ? static_cast<uint32_t>((left + 15) & ~15)
                    : rows > 0 ? static_cast<uint32_t>(rows - 1) * static_cast<uint32_t>(O.ld) +
                                     ((K + 15) & ~15)
                               : 0u;
    }
};

// This wave's share of such an image, one step of the sum: loads of 1 KB each
// straight into LDS, every WAVES-th one.  Rows, columns and elements past the matrix
// become zeros, whole 16 bytes at a time.
template <bool kCol, int W, bool kSpread, int WAVES>
struct Filler {
    static constexpr int kLoads = W / 8 / WAVES;
    static_assert(W / 8 % WAVES == 0 && WAVES % 2 == 0, "whole loads; chunks the same for all");
    uint32_t voff, ld;              // of load 0 and element 0
    int K, chunk;

    __device__ __forceinline__ Filler(const Operand &O, int K_, int wave, int lane)
        : ld(static_cast<uint32_t>(O.ld)), K(K_) {
        if constexpr (!kCol) {
            const int rho = 8 * wave + (lane >> 3);
            chunk = 16 * ((lane & 7) ^ swz_row(rho));
            voff = static_cast<uint32_t>(kSpread ? spread(rho) : rho) * ld + chunk;
        } else {
            constexpr int kChunks = W / 16, kRows = 1024 / W;
            const int k = wave * kRows + lane / kChunks;
            chunk = 16 * (lane % kChunks ^ swz_col<W>(k));
            voff = static_cast<uint32_t>(k) * ld + chunk;
        }
    }
    // load t of step s
    __device__ __forceinline__ void load(lds_char *image, const Source<kCol, W> &src, int s, int t,
                                         int wave) const {
        const int k0 = s * kBK;
        const char *b = src.base;
        uint32_t size = src.size, o;
        if constexpr (!kCol) {
            const int rows = kSpread ? spread(t * 8 * WAVES) : t * 8 * WAVES;
            o = k0 + chunk < K ? voff + (static_cast<uint32_t>(rows) * ld + k0) : kPastAll;
        } else {
            // none past the sum: no lane's place is inside its range then
            const int rows = K - k0 < kBK ? (K - k0 < 1 ? 1 : K - k0) : kBK;
            b += static_cast<uint64_t>(static_cast<uint32_t>(k0)) * ld;
            size += static_cast<uint32_t>(rows - 1) * ld;
            o = chunk < (k0 < K ? src.left : 0) ? voff + static_cast<uint32_t>(t * WAVES * (1024 / W)) * ld : kPastAll;
        }
        const __amdgpu_buffer_rsrc_t r =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(b), 0, size, 0x00020000);
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

// Of results' scales in LDS, byte x of the pair is that of this lane's row of the
// x-th 16, four of them from t and four `half` further.
__device__ __forceinline__ i32x2 spread_scales(lds_char *t, int half, int lane) {
    return read_tr(t + (lane >> 3 & 1) * half + (lane >> 1 & 3) * 16 + (lane & 1) * 8);
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

// The work of a block: tile (ti, tj) and steps [from, to) of the sum.  Blocks go
// round-robin over the 8 XCDs; each XCD takes a stretch of an order in which eight
// rows of tiles are worked off column by column, so that what its blocks read at a
// time fits its L2.
struct Item {
    int ti, tj, part, from, to;
};
__device__ __forceinline__ Item item_of(int b, int tiles_m, int tiles_n, int split, int steps) {
    constexpr int kRows = 8;
    const int tiles = tiles_m * tiles_n, n = tiles * split;
    const int xcd = b & 7, per = n >> 3, rem = n & 7;
    int t = xcd * per + (xcd < rem ? xcd : rem) + (b >> 3);
    Item o;
    o.part = split > 1 ? t / tiles : 0;
    t -= o.part * tiles;
    const int first = t / (kRows * tiles_n) * kRows;
    const int rows = tiles_m - first < kRows ? tiles_m - first : kRows;
    const int at = t - first * tiles_n;
    o.tj = at / rows;
    o.ti = first + at - o.tj * rows;
    // at most 2^15 steps, in far fewer stretches than 2^16
    o.from = static_cast<int>(static_cast<uint32_t>(steps * o.part) / static_cast<uint32_t>(split));
    o.to = static_cast<int>(static_cast<uint32_t>(steps * (o.part + 1)) / static_cast<uint32_t>(split));
    return o;
}

// Four neighbouring fp32 sums of row i from column j.
__device__ __forceinline__ void store_sums(const Out &o, int part, int i, int j, int M, int N,
                                           const f32x4 &v) {
    if (i >= M) return;
    float *p = o.sums + (static_cast<int64_t>(part) * M + i) * N + j;
    if (j + 4 <= N && (N & 3) == 0) {
        *reinterpret_cast<f32x4 *>(p) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < N) p[e] = v[e];
    }
}

// Where the scales of W results from i0 lie, four a lane and one dword a step: as they
// are, or a 128 x 128 block's one byte four times over.
struct Scales {
    const uint8_t *base;
    uint32_t step, voff, select, add, bits;
    template <int W>
    __device__ __forceinline__ void aim(const Operand &O, bool col, int i0, int lane) {
        int i = 4 * (lane % (W / 4));
        i = i0 + i < O.n ? i : (O.n - 1 - i0) & ~3;
        base = O.scales, step = 0, voff = 0, select = 0x0C0C0C0Cu, add = 0u, bits = 0u;
        if (O.blocks == FSDP_Q8_TENSOR) {       // 2^0, whatever lies there
            base = reinterpret_cast<const uint8_t *>(O.codes);
            bits = 0x7F7F7F7Fu;
        } else if (O.blocks == FSDP_Q8_TILES) {
            base += col ? i0 >> 7 : (i0 >> 7) * O.pitch;
            voff = static_cast<uint32_t>(i >> 7) * (col ? 1u : static_cast<uint32_t>(O.pitch));
            step = col ? static_cast<uint32_t>(O.pitch) : 1u, select = 0u, add = 0x01010101u;
        } else {
            base += i0;
            voff = i, step = static_cast<uint32_t>(O.pitch), select = 0x03020100u;
        }
    }
};

template <int N>
__device__ __forceinline__ void border() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// BM x BN tiles, WM x WN waves of 2 HM x 4 results of 16 x 16 each: HM rows of them in
// either half of the tile's rows.  Two images of a step in LDS, each in three parts:
// the two halves of a's rows, P0 and P1, and b's, Q.
//
// A step's products are made in two turns, one for each half.  During the first,
// P1's operands are read and the step after next's P0 and Q start on their way into
// those of this step, which were read before; during the second, the next step's P0
// is read, and its Q as the last products of the present columns are made, and P1
// of the step after next starts.  At the border after a turn every wave has the
// operands of the next turn in registers and the parts that are read in it have
// landed, two to three turns after their loads left.  (Tried before the rest stood:
// one border a step, with all loads in the second turn, took 531 us for 430 of 8192 x
// 14336 x 4096, b as it is, and 424 for 418 with b transposed.  Four waves of 128 x
// 128 in place of eight of 128 x 64 read a third less from LDS, but nothing runs
// while one of them makes addresses or waits: 465 for 400.)
//
// Eight waves keep the matrix cores busy 62% of the time, and on normal data the clock
// falls to 1.9 GHz for the card's power: 395 us, 2.4 PFLOP/s, where zeros take 315.
// Loads that all hit the caches would save 4%.
//
// A block goes from tile to tile without a pause: the last two steps of one load
// the first two of the next, and its results are stored, without a wait, before
// the next one's products.
template <int BM, int BN, int WM, int WN, bool kColA, bool kColB, int FMTA>
__global__ __launch_bounds__(64 * WM *WN, 2) void q8_product_kernel(Operand A, Operand B, Out out,
                                                                    int K) {
    constexpr int WAVES = WM * WN, HALF = BM / 2, HM = HALF / WM / 16, FN = 4, WTN = 64;
    constexpr int kStage = (BM + BN) * kBK;
    // scales in LDS: 128 bytes may be read past a wave's own
    constexpr int kScalesB = BM + 128, kScales = kScalesB + BN + 128;
    static_assert(HM * WM * 16 == HALF && HM <= 4 && BN == WN * WTN, "");
    __shared__ __attribute__((aligned(1024))) char smem[2 * kStage + 2 * kScales];
    lds_char *lds = (lds_char *)smem;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int tiles_m = (A.n + BM - 1) / BM, tiles_n = (B.n + BN - 1) / BN;
    const int items = tiles_m * tiles_n * out.split, all = (K + kBK - 1) / kBK;

    f32x4 acc[2 * HM][FN];
    auto clear = [&]() {
#pragma unroll
        for (int x = 0; x < 2 * HM; ++x)
#pragma unroll
            for (int y = 0; y < FN; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    clear();

    const Filler<kColA, HALF, false, WAVES> fa(A, K, wave, lane);
    const Filler<kColB, BN, !kColB, WAVES> fb(B, K, wave, lane);
    constexpr int kLP = decltype(fa)::kLoads, kLQ = decltype(fb)::kLoads;
    // the item that loads are for
    Item ahead = item_of(blockIdx.x, tiles_m, tiles_n, out.split, all);
    Source<kColA, HALF> src0, src1;
    Source<kColB, BN> srcq;
    // Even waves put a's scales into LDS, odd ones b's, all of them over and over: no
    // branch.
    const bool of_a = (wave & 1) == 0;
    Scales sc;
    const int db = lane % (BN / 4);
    const int sat = 2 * kStage +
                    4 * (of_a ? lane % (BM / 4) : kScalesB / 4 + (kColB ? db : spread_four(db)));
    auto aim = [&]() {
        src0.aim(A, ahead.ti * BM, K);
        src1.aim(A, ahead.ti * BM + HALF, K);
        srcq.aim(B, ahead.tj * BN, K);
        if (of_a) sc.template aim<BM>(A, kColA, ahead.ti * BM, lane);
        else sc.template aim<BN>(B, kColB, ahead.tj * BN, lane);
    };
    aim();
    // the aligned dwords that hold a step's scales, and what makes those of them
    uint32_t sw, ssel;
    auto load_scales = [&](int s) {
        const uint32_t in = s < all ? s : all - 1;
        const uint8_t *p = sc.base + static_cast<uint64_t>(in) * sc.step;
        const uint32_t low = lo32(p) & 3u;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t *>(p - low), 0, 0xFFFFFFFFu, 0x00020000);
        ssel = sc.select + ((sc.voff + low) & 3u) * sc.add;
        sw = __builtin_amdgcn_raw_buffer_load_b32(r, (sc.voff + low) & ~3u, 0, 0);
    };
    // v: the step's number in this block, over all its items
    auto put_scales = [&](int v) {
        *(lds_u32 *)(lds + sat + (v & 1) * kScales) = __builtin_amdgcn_perm(sw, sw, ssel) | sc.bits;
    };
    // What follows from the lane's number is made anew where it is used: held in
    // registers from step to step it does not fit beside the operands.
    auto anew = [&]() {
        int l = lane;
        asm volatile("" : "+v"(l));
        return l;
    };
    auto read_sa = [&](int v) {
        return spread_scales(lds + 2 * kStage + (v & 1) * kScales + wm * (HM * 16), HALF, anew());
    };
    auto read_sb = [&](int v) {
        return spread_scales(lds + 2 * kStage + (v & 1) * kScales + kScalesB + wn * WTN, 0, anew()).x;
    };
    auto part_p = [&](int v, int h) { return lds + (v & 1) * kStage + h * HALF * kBK; };
    auto part_q = [&](int v) { return lds + (v & 1) * kStage + BM * kBK; };
    auto load_p = [&](int v, int s, int h, int t) {
        fa.load(part_p(v, h), h ? src1 : src0, s, t, wave);
    };
    auto load_q = [&](int v, int s, int t) { fb.load(part_q(v), srcq, s, t, wave); };
    auto load_all = [&](int v, int s) {
#pragma unroll
        for (int t = 0; t < kLP; ++t) load_p(v, s, 0, t);
#pragma unroll
        for (int t = 0; t < kLQ; ++t) load_q(v, s, t);
#pragma unroll
        for (int t = 0; t < kLP; ++t) load_p(v, s, 1, t);
    };
    i32x8 p[2][HM], q[FN];
    auto read_p = [&](int v, int h, int x, int l) {
        if constexpr (kColA) p[h][x] = read_cols<HALF>(part_p(v, h), (wm * HM + x) * 16, l);
        else p[h][x] = read_rows(part_p(v, h), (wm * HM + x) * 16, l);
    };
    auto read_q = [&](int v, int y, int l) {
        if constexpr (kColB) q[y] = read_cols<BN>(part_q(v), wn * WTN + 16 * y, l);
        else q[y] = read_rows(part_q(v), wn * WTN + 16 * y, l);
    };
    // scales and all parts of a step: the loads younger than what a border waits for
    constexpr int kYoung = 1 + 2 * kLP + kLQ;
    static_assert(kYoung < 64, "the counter's range");
    i32x2 sa, sa2;
    int sb, sb2;
    auto mma = [&](auto hc, auto xc, auto yc) {
        constexpr int h = decltype(hc)::value, x = decltype(xc)::value, y = decltype(yc)::value;
        acc[h * HM + x][y] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            q[y], p[h][x], acc[h * HM + x][y], 0, FMTA, y, sb, x, h ? sa.y : sa.x);
    };
    // Step v.  Step s of the item that is aimed at starts on its way into the images.
    auto step = [&](int v, int s) {
        constexpr int N = HM * FN;
        int l = 0;
        // Columns outermost: the first products need the first columns alone.  Behind each
        // product what else is due, so that addresses are made while it runs (the reads'
        // ahead of a turn's first product: 411 us for 403 of 8192 x 14336 x 4096).
        for_each<N>([&](auto nc) {
            constexpr int n = decltype(nc)::value, y = n / HM, x = n % HM;
            mma(Int<0>{}, Int<x>{}, Int<y>{});
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (n == 0) {
                l = anew();
                load_scales(s);
            }
            if constexpr (n < HM) read_p(v, 1, n, l);
            constexpr int lo = n * (kLP + kLQ) / N, hi = (n + 1) * (kLP + kLQ) / N;
            for_each<hi - lo>([&](auto tc) {
                constexpr int t = lo + decltype(tc)::value;
                if constexpr (t < kLP) load_p(v + 2, s, 0, t);
                else load_q(v + 2, s, t - kLP);
            });
        });
        border<kYoung>();
        for_each<N>([&](auto nc) {
            constexpr int n = decltype(nc)::value, y = n / HM, x = n % HM;
            mma(Int<1>{}, Int<x>{}, Int<y>{});
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (n == 0) l = anew();
            if constexpr (n < HM) read_p(v + 1, 0, n, l);
            if constexpr (x == HM - 1) read_q(v + 1, y, l);
            if constexpr (n == N / 2) {
                sa2 = read_sa(v + 1);
                sb2 = read_sb(v + 1);
            }
            constexpr int lo = n * kLP / N, hi = (n + 1) * kLP / N;
            for_each<hi - lo>([&](auto tc) { load_p(v + 2, s, 1, lo + decltype(tc)::value); });
            if constexpr (n == N - 1) put_scales(v + 2);
        });
        border<kYoung>();
        sa = sa2;
        sb = sb2;
    };
    const float f = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(factor(out))));
    const bool vec = out.sums == nullptr && (B.n & 7) == 0 && (out.ld & 7) == 0 &&
                     (lo32(out.p) & 15u) == 0;
    // This lane's results of row x: twice eight neighbouring columns, from first(y).
    auto first = [&](int y, int g) {
        return wn * WTN + 32 * y + (kColB ? 16 * (g & 1) + 8 * (g >> 1) : 8 * g);
    };
    auto eight = [&](auto xc, auto yc) {
        constexpr int x = decltype(xc)::value, y = decltype(yc)::value;
        const f32x4 &a = acc[x][2 * y], &b = acc[x][2 * y + 1];
        auto two = [&](const f32x4 &c, int e) { return two_bf16(c[e] * f, c[e + 1] * f); };
        u32x4 w{two(a, 0), two(a, 2), two(b, 0), two(b, 2)};
        if constexpr (kColB) {
            // Four columns of each 16 and lane: of two lanes 16 apart, one takes the eight of
            // the first 16, the other those of the second.
            const auto s = __builtin_amdgcn_permlane16_swap(w.x, w.z, false, false);
            const auto t = __builtin_amdgcn_permlane16_swap(w.y, w.w, false, false);
            w = u32x4{s[0], t[0], s[1], t[1]};
        }
        return w;
    };
    auto results = [&](const Item &o) {
        const int i0 = o.ti * BM, j0 = o.tj * BN, l = anew(), g = l >> 4;
        if (vec) {
            // rows past the matrix lie past the range, where stores are dropped, and columns
            // past it are sent there
            const int rows = A.n - i0 < BM ? A.n - i0 : BM, cols = B.n - j0 < BN ? B.n - j0 : BN;
            const uint32_t ld = static_cast<uint32_t>(out.ld) * 2u;
            const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
                out.p + i0 * out.ld + j0, 0, static_cast<uint32_t>(rows - 1) * ld + cols * 2u,
                0x00020000);
            for_each<2 * HM>([&](auto xc) {
                constexpr int x = decltype(xc)::value;
                const uint32_t i = x / HM * HALF + (wm * HM + x % HM) * 16 + (l & 15);
                for_each<2>([&](auto yc) {
                    const int j = first(decltype(yc)::value, g);
                    const uint32_t at = j < cols ? i * ld + j * 2u : 0xFFFFFFF0u;
                    __builtin_amdgcn_raw_buffer_store_b128(eight(xc, yc), r, at, 0, 0);
                });
            });
            return;
        }
        for_each<2 * HM>([&](auto xc) {
            constexpr int x = decltype(xc)::value;
            const int i = i0 + x / HM * HALF + (wm * HM + x % HM) * 16 + (l & 15);
            if (out.sums != nullptr) {
                // fours of columns, as they come
                for_each<FN>([&](auto yc) {
                    constexpr int y = decltype(yc)::value;
                    const int j = j0 + wn * WTN +
                                  (kColB ? 16 * y + 4 * g : 32 * (y >> 1) + 8 * g + 4 * (y & 1));
                    store_sums(out, o.part, i, j, A.n, B.n, acc[x][y]);
                });
            } else {
                for_each<2>([&](auto yc) {
                    const u32x4 w = eight(xc, yc);
                    const int j = j0 + first(decltype(yc)::value, g);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (i < A.n && j + e < B.n)
                            out.p[i * out.ld + j + e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
                });
            }
        });
    };

    // Loads for steps that no item has read nothing, and are counted.
    Item now = ahead;
    load_scales(now.from);
    load_all(0, now.from);
    put_scales(0);
    load_scales(now.from + 1);
    load_all(1, now.from + 1);
    put_scales(1);
    border<2 * kLP + kLQ>();
    sa = read_sa(0);
    sb = read_sb(0);
#pragma unroll
    for (int x = 0; x < HM; ++x) read_p(0, 0, x, lane);
#pragma unroll
    for (int y = 0; y < FN; ++y) read_q(0, y, lane);
    border<2 * kLP + kLQ>();
    int v = 0;
    for (int b = blockIdx.x;;) {
        int s = now.from;
        for (; s + 2 < now.to; ++s, ++v) step(v, s + 2);
        b += gridDim.x;
        if (b < items) ahead = item_of(b, tiles_m, tiles_n, out.split, all);
        else ahead.from = all;
        aim();
        for (int i = 0; s < now.to; ++s, ++v, ++i) step(v, ahead.from + i);
        results(now);
        if (b >= items) break;
        clear();
        now = ahead;
    }
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------

// Up to 16 FM rows by b transposed: b is read once, which bounds the time (58.7 MB for
// one row by 14336 x 4096), and nothing in LDS would be read twice.  A block has 16 FN
// columns, and each of its eight waves every eighth step of the sum, so that many
// loads are under way however few columns there are; the waves' sums meet in LDS, in
// their order.
constexpr int kFewWaves = 8;

// The scale of a row at step s, one byte.
__device__ __forceinline__ int few_scale(const Operand &O, int i, int s) {
    if (O.blocks == FSDP_Q8_TENSOR) return 127;
    const int64_t at = O.blocks == FSDP_Q8_TILES ? (i >> 7) * O.pitch + s
                                                 : static_cast<int64_t>(s) * O.pitch + i;
    return O.scales[at];
}

template <int FM, int FN, int FMTA>
__global__ __launch_bounds__(64 * kFewWaves) void q8_few_kernel(Operand A, Operand B, Out out, int K) {
    __shared__ __attribute__((aligned(16))) f32x4 sums[kFewWaves][FM * FN][64];
    const int tid = threadIdx.x, lane = tid & 63, j = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j0 = blockIdx.x * 16 * FN, steps = (K + kBK - 1) / kBK;
    // rows past the matrix are read as its last one; what comes of them is dropped
    const char *row_a[FM], *row_b[FN];
    int ia[FM], ib[FN];
#pragma unroll
    for (int x = 0; x < FM; ++x) {
        ia[x] = 16 * x + j < A.n ? 16 * x + j : A.n - 1;
        row_a[x] = A.codes + ia[x] * A.ld;
    }
#pragma unroll
    for (int y = 0; y < FN; ++y) {
        ib[y] = j0 + 16 * y + j < B.n ? j0 + 16 * y + j : B.n - 1;
        row_b[y] = B.codes + ib[y] * B.ld;
    }
    struct Step {
        Frag a[FM], b[FN];
        int sa[FM], sb[FN];
    };
    // chunks past the sum are zeros
    auto load = [&](Step &t, int s) {
        const int k = s * kBK + 16 * g;
        const bool in0 = k < K, in1 = k + 64 < K;
        const int k1 = in1 ? k + 64 : 0, kk = in0 ? k : 0;
        auto one = [&](const char *row) {
            Frag f;
            f.h[0] = *reinterpret_cast<const i32x4 *>(row + kk);
            f.h[1] = *reinterpret_cast<const i32x4 *>(row + k1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f.h[0][e] = in0 ? f.h[0][e] : 0;
                f.h[1][e] = in1 ? f.h[1][e] : 0;
            }
            return f;
        };
#pragma unroll
        for (int y = 0; y < FN; ++y) t.b[y] = one(row_b[y]), t.sb[y] = few_scale(B, ib[y], s);
#pragma unroll
        for (int x = 0; x < FM; ++x) t.a[x] = one(row_a[x]), t.sa[x] = few_scale(A, ia[x], s);
    };
    f32x4 acc[FM][FN];
#pragma unroll
    for (int x = 0; x < FM; ++x)
#pragma unroll
        for (int y = 0; y < FN; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // two steps' loads at a time
    for (int s = wave; s < steps; s += 2 * kFewWaves) {
        Step t[2];
        const int s1 = s + kFewWaves < steps ? s + kFewWaves : s;
        load(t[0], s);
        load(t[1], s1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h == 1 && s1 == s) break;
#pragma unroll
            for (int x = 0; x < FM; ++x)
#pragma unroll
                for (int y = 0; y < FN; ++y)
                    acc[x][y] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        t[h].b[y].v, t[h].a[x].v, acc[x][y], 0, FMTA, 0, t[h].sb[y], 0, t[h].sa[x]);
        }
    }
#pragma unroll
    for (int x = 0; x < FM; ++x)
#pragma unroll
        for (int y = 0; y < FN; ++y) sums[wave][x * FN + y][lane] = acc[x][y];
    __syncthreads();
    // Row 16 x + j of the results, columns 4 g .. + 4 of the y-th 16.
    const float f = factor(out);
    for (int u = tid; u < FM * FN * 64; u += 64 * kFewWaves) {
        const int n = u >> 6, l = u & 63;
        f32x4 v = sums[0][n][l];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) v += sums[w][n][l];
        const int i = n / FN * 16 + (l & 15), c = j0 + n % FN * 16 + (l >> 4) * 4;
        if (i >= A.n) continue;
        uint16_t *p = out.p + i * out.ld + c;
        const uint32_t lo = two_bf16(v[0] * f, v[1] * f), hi = two_bf16(v[2] * f, v[3] * f);
        if (c + 4 <= B.n && (lo32(out.p) & 7u) == 0 && (out.ld & 3) == 0) {
            *reinterpret_cast<u32x2 *>(p) = u32x2{lo, hi};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < B.n) p[e] = static_cast<uint16_t>((e < 2 ? lo : hi) >> (16 * (e & 1)));
        }
    }
}

// The stretches' sums in order, four neighbouring results a thread where rows are
// whole fours.
template <int n>
__global__ __launch_bounds__(kBlock) void q8_join_kernel(Out out, int M, int N) {
    typedef float vec __attribute__((ext_vector_type(n)));
    const int64_t all = static_cast<int64_t>(M) * N / n;
    const float f = factor(out);
    const vec *sums = reinterpret_cast<const vec *>(out.sums);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < all;
         i += static_cast<int64_t>(gridDim.x) * kBlock) {
        vec s = sums[i];
        for (int k = 1; k < out.split; ++k) s += sums[k * all + i];
        const int64_t row = i * n / N;
        uint16_t *p = out.p + row * out.ld + (i * n - row * N);
#pragma unroll
        for (int e = 0; e < n; ++e) p[e] = static_cast<uint16_t>(two_bf16(s[e] * f, 0.0f));
    }
}

// An empty sum.
__global__ __launch_bounds__(kBlock) void q8_zero_kernel(Out out, int M, int N) {
    const int64_t n = static_cast<int64_t>(M) * N;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kBlock) {
        const int64_t row = i / N;
        out.p[row * out.ld + (i - row * N)] = 0;
    }
}

// Rows of any alignment to rows of whole 16 bytes, zeros after their end.
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
    // Blocks that fit the device at once go on from item to item, if every item has the
    // two steps that load the next one's.
    constexpr int kAtOnce = 256 * (163840 / (2 * (BM + BN) * kBK + 4096));
    const int items = (A.n + BM - 1) / BM * ((B.n + BN - 1) / BN) * out.split;
    const int steps = (K + kBK - 1) / kBK;
    const int grid = items > kAtOnce && steps / out.split >= 2 ? kAtOnce : items;
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

template <int FM, int FN>
void launch_few(const Operand &A, const Operand &B, int format, const Out &out, int K,
                hipStream_t st) {
    const int grid = (B.n + 16 * FN - 1) / (16 * FN);
    void (*kernel)(Operand, Operand, Out, int) =
        format == FSDP_Q8_E4M3 ? q8_few_kernel<FM, FN, 0> : q8_few_kernel<FM, FN, 1>;
    kernel<<<grid, 64 * kFewWaves, 0, st>>>(A, B, out, K);
}

int64_t round16(int64_t x) { return (x + 15) & ~int64_t{15}; }

}  // namespace

hipError_t launch_q8_product(const Q8Mat &a, bool ta, const Q8Mat &b, bool tb, uint16_t *p,
                             int64_t ldo, const Q8Cut &cut, void *ws, hipStream_t st) {
    const int M = ta ? a.cols : a.rows, N = tb ? b.rows : b.cols, K = ta ? a.rows : a.cols;
    if (M == 0 || N == 0) return hipSuccess;
    if (K == 0) {
        q8_zero_kernel<<<blocks_for(static_cast<int64_t>(M) * N), kBlock, 0, st>>>(
            Out{p, nullptr, nullptr, nullptr, ldo, 1}, M, N);
        return hipGetLastError();
    }
    char *at = static_cast<char *>(ws);
    auto operand = [&](const Q8Mat &m, int64_t bytes, int n) {
        Operand o{reinterpret_cast<const char *>(m.codes), m.scales, m.ld, m.pitch, n, m.blocks};
        if (bytes > 0) {
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
    if (cut.tile == 0) {
        launch<256, 256, 2, 4>(A, ta, B, tb, a.format, out, K, st);
    } else if (cut.tile == 1) {
        launch<128, 128, 2, 2>(A, ta, B, tb, a.format, out, K, st);
    } else if (cut.tile == 2) {
        launch<64, 64, 2, 1>(A, ta, B, tb, a.format, out, K, st);
    } else {
        // Columns a block: 16 while every CU has at most one such block, then 32 (K = 4096, one
        // row and 32: 4096 columns 4.9 us for 6.8 and 7.9 for 9.9 with 32, 4112 6.8 either way
        // and 10.3 for 13.3 with 16, 8192 7.0 for 7.4 and 10.4 for 14.0, 14336 12.9 for 13.8 and
        // 18.3 for 25.2; of one row by 8193 to 12288, three turns for two, 16 would take 9.5
        // to 10.0 for 10.9).
        const bool wide = N > 16 * 256;
        if (M <= 16) wide ? launch_few<1, 2>(A, B, a.format, out, K, st)
                          : launch_few<1, 1>(A, B, a.format, out, K, st);
        else wide ? launch_few<2, 2>(A, B, a.format, out, K, st)
                  : launch_few<2, 1>(A, B, a.format, out, K, st);
    }
    if (cut.split > 1) {
        const int64_t n = static_cast<int64_t>(M) * N;
        if (N % 4 == 0) q8_join_kernel<4><<<blocks_for(n / 4), kBlock, 0, st>>>(out, M, N);
        else q8_join_kernel<1><<<blocks_for(n), kBlock, 0, st>>>(out, M, N);
    }
    return hipGetLastError();
}

}  // namespace fsdp
