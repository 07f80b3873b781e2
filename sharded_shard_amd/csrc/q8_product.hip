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

__device__ __forceinline__ void load_lds(const char *base, uint32_t nbytes, uint32_t voff,
                                         lds_char *to) {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(base), 0, nbytes, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)to, 16, voff, 0, 0, 0);
}

// Load u (1 KB) of an operand's image for the step from element k0 of the sum.
// Rows, columns and elements past the matrix become zeros, whole 16 bytes at a
// time.
template <bool kCol, int W, bool kSpread>
__device__ __forceinline__ void fill(lds_char *dst, const Operand &O, int i0, int k0, int K, int u,
                                     int lane) {
    if constexpr (!kCol) {
        const int rho = 8 * u + (lane >> 3), c = (lane & 7) ^ swz_row(rho);
        const int row = kSpread ? spread(rho) : rho, left = O.n - i0;
        const bool in = row < left && k0 + 16 * c < K;
        const uint32_t voff = static_cast<uint32_t>(row) * static_cast<uint32_t>(O.ld) + k0 + 16 * c;
        const int rows = left < W ? left : W;
        const uint32_t nbytes =
            static_cast<uint32_t>(rows - 1) * static_cast<uint32_t>(O.ld) + ((K + 15) & ~15);
        load_lds(O.codes + static_cast<int64_t>(i0) * O.ld, nbytes, in ? voff : kPastAll,
                 dst + u * 1024);
    } else {
        constexpr int kChunks = W / 16, kRows = 1024 / W;
        const int k = u * kRows + lane / kChunks, c = lane % kChunks ^ swz_col<W>(k);
        const int left = O.n - i0;
        const bool in = k0 + k < K && 16 * c < left;
        const uint32_t voff = static_cast<uint32_t>(k) * static_cast<uint32_t>(O.ld) + 16 * c;
        const int rows = K - k0 < kBK ? K - k0 : kBK;
        const uint32_t nbytes =
            static_cast<uint32_t>(rows - 1) * static_cast<uint32_t>(O.ld) + ((left + 15) & ~15);
        load_lds(O.codes + static_cast<int64_t>(k0) * O.ld + i0, nbytes, in ? voff : kPastAll,
                 dst + u * 1024);
    }
}

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

// Scales of step kb for four results from i, i a multiple of 4.
template <bool kCol>
__device__ __forceinline__ uint32_t load_scales(const Operand &O, int kb, int i) {
    if (O.blocks == FSDP_Q8_TENSOR || i >= O.n) return 0x7F7F7F7Fu;
    if (O.blocks == FSDP_Q8_TILES) {
        const int64_t at = kCol ? static_cast<int64_t>(kb) * O.pitch + (i >> 7)
                                : static_cast<int64_t>(i >> 7) * O.pitch + kb;
        return O.scales[at] * 0x01010101u;
    }
    return *reinterpret_cast<const uint32_t *>(O.scales + static_cast<int64_t>(kb) * O.pitch + i);
}

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

// n neighbouring results of row i from column j.
template <int n, typename F>
__device__ __forceinline__ void store(const Out &o, float f, int i, int j, int M, int N, F &&get) {
    if (o.sums != nullptr) {
        float *p = o.sums + (static_cast<int64_t>(blockIdx.z) * M + i) * N + j;
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

template <int BM, int BN, int WM, int WN, bool kColA, bool kColB, int FMTA>
__global__ __launch_bounds__(64 * WM *WN) void q8_product_kernel(Operand A, Operand B, Out out,
                                                                 int K) {
    constexpr int WAVES = WM * WN, WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
    constexpr int kScales = (BM < 128 ? 128 : BM) + (BN < 128 ? 128 : BN) + 128;
    constexpr int kStage = (BM + BN) * kBK;
    static_assert(FN % 4 == 0 && FM <= 8 && FN <= 8, "");
    __shared__ __attribute__((aligned(1024))) char smem[2 * kStage + 2 * kScales];
    lds_char *lds = (lds_char *)smem;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN, g = lane >> 4;
    const int i0 = blockIdx.x * BM, j0 = blockIdx.y * BN;
    const int all = (K + kBK - 1) / kBK;
    const int from = static_cast<int>(static_cast<int64_t>(all) * blockIdx.z / out.split);
    const int to = static_cast<int>(static_cast<int64_t>(all) * (blockIdx.z + 1) / out.split);

    auto image = [&](int s) { return lds + (s & 1) * kStage; };
    auto scales = [&](int s) { return lds + 2 * kStage + (s & 1) * kScales; };
    constexpr int kScalesB = BM < 128 ? 128 : BM;
    auto fill_step = [&](int s) {
#pragma unroll
        for (int u = 0; u < (BM / 8 + WAVES - 1) / WAVES; ++u)
            if (u * WAVES + wave < BM / 8)
                fill<kColA, BM, false>(image(s), A, i0, s * kBK, K, u * WAVES + wave, lane);
#pragma unroll
        for (int u = 0; u < (BN / 8 + WAVES - 1) / WAVES; ++u)
            if (u * WAVES + wave < BN / 8)
                fill<kColB, BN, !kColB>(image(s) + BM * kBK, B, j0, s * kBK, K, u * WAVES + wave,
                                        lane);
    };
    const int tid = threadIdx.x;
    auto step_scales = [&](int s) {
        if (tid < BM / 4) return load_scales<kColA>(A, s, i0 + 4 * tid);
        if (tid < BM / 4 + BN / 4) return load_scales<kColB>(B, s, j0 + 4 * (tid - BM / 4));
        return 0u;
    };

    f32x4 acc[FM][FN];
#pragma unroll
    for (int x = 0; x < FM; ++x)
#pragma unroll
        for (int y = 0; y < FN; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    if (from < to) fill_step(from);
    uint32_t sc = from < to ? step_scales(from) : 0u;
    for (int s = from; s < to; ++s) {
        if (tid < BM / 4 + BN / 4)
            *(lds_u32 *)(scales(s) + (tid < BM / 4 ? 4 * tid : kScalesB + 4 * (tid - BM / 4))) = sc;
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (s + 1 < to) {
            fill_step(s + 1);
            sc = step_scales(s + 1);
        }
        lds_char *ta = image(s), *tb = ta + BM * kBK;
        if ((!kColA || !kColB) && s == all - 1 && (K & 15) != 0) {
            // what follows the sum's last element in its 16 bytes is no part of it
            const int c = (K & 127) >> 4, keep = K & 15;
            for (int r = tid; r < (kColA ? 0 : BM) + (kColB ? 0 : BN); r += 64 * WAVES) {
                const int row = !kColA && r < BM ? r : r - (kColA ? 0 : BM);
                lds_char *p = (!kColA && r < BM ? ta : tb) + row * 128 + (c ^ swz_row(row)) * 16;
                for (int b = keep; b < 16; ++b) p[b] = 0;
            }
            __syncthreads();
        }
        i32x8 p[FM], q[FN];
        const i32x2 sa = spread_scales(scales(s) + wm * WTM, lane);
        int sb[2];
        if constexpr (kColB) {
            const i32x2 t = spread_scales(scales(s) + kScalesB + wn * WTN, lane);
            sb[0] = t.x;
            sb[1] = t.y;
        } else {
#pragma unroll
            for (int h = 0; h < FN / 4; ++h)
                sb[h] = *(const lds_u32 *)(scales(s) + kScalesB + wn * WTN + 64 * h + 4 * (lane & 15));
        }
#pragma unroll
        for (int x = 0; x < FM; ++x) {
            if constexpr (kColA) p[x] = read_cols<BM>(ta, wm * WTM + 16 * x, lane);
            else p[x] = read_rows(ta, wm * WTM + 16 * x, lane);
        }
#pragma unroll
        for (int y = 0; y < FN; ++y) {
            if constexpr (kColB) q[y] = read_cols<BN>(tb, wn * WTN + 16 * y, lane);
            else q[y] = read_rows(tb, wn * WTN + 16 * y, lane);
        }
        auto mma = [&](auto xc, auto yc) {
            constexpr int x = decltype(xc)::value, y = decltype(yc)::value;
            acc[x][y] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                q[y], p[x], acc[x][y], 0, FMTA, y & 3, sb[y >> 2], x & 3, x < 4 ? sa.x : sa.y);
        };
        for_each<FM>([&](auto xc) { for_each<FN>([&](auto yc) { mma(xc, yc); }); });
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
                    store<4>(out, f, i, j0 + wn * WTN + 16 * y + 4 * g, A.n, B.n,
                             [&](int e) { return acc[x][y][e]; });
                });
            } else {
                for_each<FN / 4>([&](auto hc) {
                    constexpr int h = decltype(hc)::value;
                    store<16>(out, f, i, j0 + wn * WTN + 64 * h + 16 * g, A.n, B.n,
                              [&](int e) { return acc[x][4 * h + (e & 3)][e >> 2]; });
                });
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
    const dim3 grid((A.n + BM - 1) / BM, (B.n + BN - 1) / BN, out.split);
    constexpr int kThreads = 64 * WM * WN;
    auto go = [&](auto kernel) { kernel<<<grid, kThreads, 0, st>>>(A, B, out, K); };
    const bool e4 = format == FSDP_Q8_E4M3;
    if (!ta && tb)
        e4 ? go(q8_product_kernel<BM, BN, WM, WN, false, false, 0>)
           : go(q8_product_kernel<BM, BN, WM, WN, false, false, 1>);
    else if (!ta)
        e4 ? go(q8_product_kernel<BM, BN, WM, WN, false, true, 0>)
           : go(q8_product_kernel<BM, BN, WM, WN, false, true, 1>);
    else
        e4 ? go(q8_product_kernel<BM, BN, WM, WN, true, true, 0>)
           : go(q8_product_kernel<BM, BN, WM, WN, true, true, 1>);
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
    c.tile = M <= 64 || N <= 64 ? 1 : 0;
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
    if (cut.tile == 0) launch<128, 128, 2, 2>(A, ta, B, tb, a.format, out, K, st);
    else launch<64, 64, 2, 1>(A, ta, B, tb, a.format, out, K, st);
    if (cut.split > 1)
        q8_join_kernel<<<blocks_for(static_cast<int64_t>(M) * N), kBlock, 0, st>>>(out, M, N);
    return hipGetLastError();
}

}  // namespace fsdp
