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
#include "q8_device.hpp"

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

// x over a caller's scale, which may leave it past fmax, or past fp32: clamped there;
// the comparisons keep NaN.  x - x is 0, or NaN where x is not finite: an infinity is
// no value that a code could stand in for.  It is subtracted, since -0 - 0 is -0 (-0 + 0
// is not).
__device__ __forceinline__ float clamped(float x, float inverse) {
    const float y = x * inverse;
    return (y > 448.0f ? 448.0f : (y < -448.0f ? -448.0f : y)) - (x - x);
}

// Four codes of values that fit.
template <int FMT>
__device__ __forceinline__ uint32_t four_codes(float a, float b, float c, float d) {
    int w;
    if constexpr (FMT == FSDP_Q8_E4M3) {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    }
    return static_cast<uint32_t>(w);
}

typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// Four codes of four bf16 over a power of two, one instruction for two (equal to the
// converter of fp32 on the quotient for every bf16 that fits and every scale).
template <int FMT>
__device__ __forceinline__ uint32_t four_scaled(uint32_t lo, uint32_t hi, float s) {
    s16x2 w{0, 0};
    const bf16x2 a = __builtin_bit_cast(bf16x2, lo), b = __builtin_bit_cast(bf16x2, hi);
    if constexpr (FMT == FSDP_Q8_E4M3) {
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, a, s, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, b, s, true);
    } else {
        w = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(w, a, s, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(w, b, s, true);
    }
    return __builtin_bit_cast(uint32_t, w);
}

// Both halves' maxima.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
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

// The maximum over 16 neighbouring lanes, in each of them, by rotating them.
template <bool kHalves>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    auto step = [&](uint32_t o) { v = kHalves ? max2(v, o) : umax(v, o); };
    step(__builtin_amdgcn_update_dpp(0u, v, 0x128, 0xF, 0xF, false));
    step(__builtin_amdgcn_update_dpp(0u, v, 0x124, 0xF, 0xF, false));
    step(__builtin_amdgcn_update_dpp(0u, v, 0x122, 0xF, 0xF, false));
    step(__builtin_amdgcn_update_dpp(0u, v, 0x121, 0xF, 0xF, false));
    return v;
}

// The maximum over the wave's four lanes 16 apart, in each of them.
template <bool kHalves>
__device__ __forceinline__ uint32_t column_max(uint32_t v) {
    auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = kHalves ? max2(a[0], a[1]) : umax(a[0], a[1]);
    a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return kHalves ? max2(a[0], a[1]) : umax(a[0], a[1]);
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

// One 128 x 128 block a workgroup, held in registers from the loads to the stores:
// thread (r, c) of 128 / P x 16 has the eight columns from 8 c of P rows.  A row's
// maximum is taken over its 16 neighbouring lanes, a column's over the wave's four
// rows and, through LDS, over the waves.
//
// Of bf16 the magnitudes are compared two at a time as 16-bit numbers, and one
// instruction divides two by their scale and rounds them.  The scales of two
// neighbouring columns differ, but are powers of two: their exponents, less that of a
// common scale 2^(kLow - 127), are taken from the values', two at a time, and what
// is left is over the common one.  A value that this leaves under 2^-126 is under
// 2^-22 of its scale, no code's worth, and may come out as anything as small.
// (8192 x 4096 both ways: 39 us with a product and a conversion from fp32 for each
// value.)
constexpr uint32_t kLow = 24;

template <int FMT, bool kF32, int WHAT, int P>
__global__ __launch_bounds__(2048 / P) void q8_quantize_kernel(const void *__restrict__ x,
                                                               int64_t ldx, Q8Mat A, Q8Mat B) {
    constexpr int kWaves = 32 / P, kRows = 128 / P, kWords = kF32 ? 8 : 4;
    __shared__ __attribute__((aligned(16))) uint32_t part[kWaves][16][kWords];
    __shared__ __attribute__((aligned(16))) uint8_t bytes[2][128];
    const int tid = threadIdx.x, r = tid >> 4, t16 = tid & 15, c = t16 * 8, wave = tid >> 6;
    const int row0 = blockIdx.y * 128, col0 = blockIdx.x * 128;
    const int rows = A.rows - row0 < 128 ? A.rows - row0 : 128;
    const int cols = A.cols - col0 < 128 ? A.cols - col0 : 128;
    const int n = cols - c < 0 ? 0 : (cols - c < 8 ? cols - c : 8);
    const bool vec = (lo32(x) & 15u) == 0 && (ldx & (kF32 ? 3 : 7)) == 0;
    const Q8Mat &rm = A, &cm = (WHAT & kWriteRows) && (WHAT & kWriteCols) ? B : A;
    Eight<kF32> v[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int row = r + kRows * p;
        const int64_t o = static_cast<int64_t>(row0 + row) * ldx + col0 + c;
        v[p] = load_eight<kF32>(x, o, row < rows ? n : 0, vec);
    }
    // magnitudes, two in a word of bf16; what is not finite has none
    uint32_t mag[P][kWords];
    bool odd = false;
    if constexpr (kF32) {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int e = 0; e < 8; ++e) mag[p][e] = finite_mag(v[p].get(e));
    } else {
        uint32_t most = 0;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mag[p][e] = v[p].w[0][e] & 0x7FFF7FFFu;
                most = max2(most, mag[p][e]);
            }
        odd = __any((most & 0xFFFFu) >= 0x7F80u || (most >> 16) >= 0x7F80u);
        if (odd) {
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t m = mag[p][e];
                    mag[p][e] = ((m & 0xFFFFu) < 0x7F80u ? m & 0xFFFFu : 0u) |
                                (m < 0x7F800000u ? m & 0xFFFF0000u : 0u);
                }
        }
    }
    auto codes_at = [&](const Q8Mat &m, int row) {
        return m.codes + static_cast<int64_t>(row0 + row) * m.ld + col0 + c;
    };
    // row p over one scale for all its values
    auto put_row = [&](const Q8Mat &m, bool wide, int p, uint32_t byte) {
        const int row = r + kRows * p;
        uint32_t lo, hi;
        if constexpr (kF32) {
            const float s = inverse_scale(byte);
            lo = four_codes<FMT>(v[p].get(0) * s, v[p].get(1) * s, v[p].get(2) * s, v[p].get(3) * s);
            hi = four_codes<FMT>(v[p].get(4) * s, v[p].get(5) * s, v[p].get(6) * s, v[p].get(7) * s);
        } else {
            const float s = scale_of(byte);
            lo = four_scaled<FMT>(v[p].w[0].x, v[p].w[0].y, s);
            hi = four_scaled<FMT>(v[p].w[0].z, v[p].w[0].w, s);
        }
        if (row < rows) store_eight(codes_at(m, row), lo, hi, n, wide);
    };
    if constexpr (WHAT & kWriteRows) {
        const bool wide = (lo32(rm.codes) & 7u) == 0 && (rm.ld & 7) == 0;
        auto put = [&](int p, uint32_t m) {
            const uint32_t b = scale_byte<FMT>(m);
            if (t16 == 0) bytes[0][r + kRows * p] = static_cast<uint8_t>(b);
            put_row(rm, wide, p, b);
        };
        if constexpr (kF32) {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) m = umax(m, mag[p][e]);
                put(p, row_max<false>(m));
            }
        } else {
#pragma unroll
            for (int p = 0; p < P; p += 2) {
                auto four = [&](int k) {
                    return max2(max2(mag[k][0], mag[k][1]), max2(mag[k][2], mag[k][3]));
                };
                // two rows' maxima in the halves of a word
                const uint32_t a = four(p), b = four(p + 1);
                const uint32_t m = row_max<true>(max2(__builtin_amdgcn_perm(b, a, 0x05040100u),
                                                      __builtin_amdgcn_perm(b, a, 0x07060302u)));
                put(p, m << 16);
                put(p + 1, m & 0xFFFF0000u);
            }
        }
    }
    if constexpr (WHAT & (kWriteCols | kWriteTiles)) {
#pragma unroll
        for (int e = 0; e < kWords; ++e) {
            uint32_t m = 0;
#pragma unroll
            for (int p = 0; p < P; ++p) m = kF32 ? umax(m, mag[p][e]) : max2(m, mag[p][e]);
            m = column_max<!kF32>(m);
            if ((tid & 48) == 0) part[wave][t16][e] = m;
        }
    }
    __syncthreads();
    if constexpr (WHAT & (kWriteCols | kWriteTiles)) {
        const bool wide = (lo32(cm.codes) & 7u) == 0 && (cm.ld & 7) == 0;
        uint32_t m[kWords];
#pragma unroll
        for (int e = 0; e < kWords; ++e) m[e] = part[0][t16][e];
#pragma unroll
        for (int w = 1; w < kWaves; ++w)
#pragma unroll
            for (int e = 0; e < kWords; ++e)
                m[e] = kF32 ? umax(m[e], part[w][t16][e]) : max2(m[e], part[w][t16][e]);
        if constexpr (WHAT & kWriteTiles) {
            uint32_t all = 0;
#pragma unroll
            for (int e = 0; e < kWords; ++e) all = kF32 ? umax(all, m[e]) : max2(all, m[e]);
            all = row_max<!kF32>(all);
            if constexpr (!kF32) all = umax(all << 16, all & 0xFFFF0000u);
            const uint32_t b = scale_byte<FMT>(all);
            if (tid == 0)
                cm.scales[static_cast<int64_t>(blockIdx.y) * cm.pitch + blockIdx.x] =
                    static_cast<uint8_t>(b);
#pragma unroll
            for (int p = 0; p < P; ++p) put_row(cm, wide, p, b);
        } else {
            uint32_t b[8];
            bool low = odd;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t k = kF32 ? m[e] : e & 1 ? m[e >> 1] & 0xFFFF0000u : m[e >> 1] << 16;
                b[e] = scale_byte<FMT>(k);
                low |= k != 0 && b[e] < kLow;
                if (r == 0) bytes[1][c + e] = static_cast<uint8_t>(b[e]);
            }
            if (kF32 || __any(low)) {
                float s[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = inverse_scale(b[e]);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const int row = r + kRows * p;
                    if (row < rows)
                        store_eight(codes_at(cm, row),
                                    four_codes<FMT>(v[p].get(0) * s[0], v[p].get(1) * s[1],
                                                    v[p].get(2) * s[2], v[p].get(3) * s[3]),
                                    four_codes<FMT>(v[p].get(4) * s[4], v[p].get(5) * s[5],
                                                    v[p].get(6) * s[6], v[p].get(7) * s[7]),
                                    n, wide);
                }
            } else {
                // an empty column's zeros stay zeros
                uint32_t less[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t lo = b[2 * e] < kLow ? 0u : b[2 * e] - kLow;
                    const uint32_t hi = b[2 * e + 1] < kLow ? 0u : b[2 * e + 1] - kLow;
                    less[e] = lo << 7 | hi << 23;
                }
                const float s = scale_of(kLow);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    const int row = r + kRows * p;
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const u16x2 d = __builtin_elementwise_sub_sat(
                            __builtin_bit_cast(u16x2, mag[p][e]), __builtin_bit_cast(u16x2, less[e]));
                        w[e] = (v[p].w[0][e] & 0x80008000u) | __builtin_bit_cast(uint32_t, d);
                    }
                    if (row < rows)
                        store_eight(codes_at(cm, row), four_scaled<FMT>(w[0], w[1], s),
                                    four_scaled<FMT>(w[2], w[3], s), n, wide);
                }
            }
            __syncthreads();
        }
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
template <int FMT, bool kF32, int P, bool kDiv>
__global__ __launch_bounds__(2048 / P) void q8_dequantize_kernel(Q8Mat Q, void *__restrict__ out,
                                                                 int64_t ldo) {
    constexpr int kRows = 128 / P;
    const int tid = threadIdx.x, r = tid >> 4, c = (tid & 15) * 8;
    const int row0 = blockIdx.y * 128, col0 = blockIdx.x * 128;
    const int rows = Q.rows - row0 < 128 ? Q.rows - row0 : 128;
    const int cols = Q.cols - col0 < 128 ? Q.cols - col0 : 128;
    const int n = cols - c < 0 ? 0 : (cols - c < 8 ? cols - c : 8);
    if (n == 0) return;
    const bool vec = n == 8 && (lo32(Q.codes) & 7u) == 0 && (Q.ld & 7) == 0;
    const bool wide = n == 8 && (lo32(out) & 15u) == 0 && (ldo & (kF32 ? 3 : 7)) == 0;
    const float div = kDiv ? *Q.divisor : 1.0f;
    // All loads leave before the first is waited for: rows past the matrix read its first
    // again.
    uint32_t w[P][2];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int row = r + kRows * p < rows ? r + kRows * p : 0;
        const uint8_t *from = Q.codes + static_cast<int64_t>(row0 + row) * Q.ld + col0 + c;
        if (vec) {
            const u32x2 t = *reinterpret_cast<const u32x2 *>(from);
            w[p][0] = t.x;
            w[p][1] = t.y;
        } else {
            w[p][0] = w[p][1] = 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) w[p][e >> 2] |= static_cast<uint32_t>(from[e]) << (8 * (e & 3));
        }
    }
    uint32_t by_row[P], by_col[8];
    const uint8_t *sb = Q.scales + static_cast<int64_t>(Q.blocks == FSDP_Q8_ROWS ? blockIdx.x
                                                                                : blockIdx.y) *
                                       Q.pitch;
#pragma unroll
    for (int p = 0; p < P; ++p) by_row[p] = 127u;
#pragma unroll
    for (int e = 0; e < 8; ++e) by_col[e] = 127u;
    if (Q.blocks == FSDP_Q8_ROWS) {
#pragma unroll
        for (int p = 0; p < P; ++p) by_row[p] = sb[row0 + (r + kRows * p < rows ? r + kRows * p : 0)];
    } else if (Q.blocks == FSDP_Q8_COLS) {
        if (n == 8) {
            // a line starts at a multiple of four bytes
            const uint32_t *q = reinterpret_cast<const uint32_t *>(sb + col0 + c);
            const uint32_t lo = q[0], hi = q[1];
#pragma unroll
            for (int e = 0; e < 8; ++e) by_col[e] = (e < 4 ? lo : hi) >> (8 * (e & 3)) & 255u;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) by_col[e] = sb[col0 + c + (e < n ? e : 0)];
        }
    } else if (Q.blocks == FSDP_Q8_TILES) {
        const uint32_t b = sb[blockIdx.x];
#pragma unroll
        for (int p = 0; p < P; ++p) by_row[p] = b;
    }
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = scale_of(by_col[e]);
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int row = r + kRows * p;
        if (row >= rows) continue;
        const float sr = scale_of(by_row[p]);
        float y[8];
        code_values<FMT>(w[p][0], w[p][1], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // one of the two is 1
            y[e] *= Q.blocks == FSDP_Q8_COLS ? s[e] : sr;
            if constexpr (kDiv) y[e] /= div;
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
            u32x4 h;
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = two_bf16(y[2 * e], y[2 * e + 1]);
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
// four each, without keeping them in the caches.  Of a decoder block's shards on 8 ranks,
// 122 MB, that takes 22 us for 24, and with the copy-in right after it, which then reads
// them from memory, 55 for 54; with 512 MB of other work's writes between the two, as a
// step has its collective there, 68 for 88.  Cells of entry -1 are blocks that other ranks
// hold alone: zeros.
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
                const f32x4 v = ldp<1>(reinterpret_cast<const f32x4 *>(p + r * width + c));
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
            const float v = clamped(src[i], scale_at(place_after(row0, col0, i, be.cols)));
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
                    w[k] = four_codes<FSDP_Q8_E4M3>(clamped(v[k].x, s), clamped(v[k].y, s),
                                                    clamped(v[k].z, s), clamped(v[k].w, s));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        y[e] = clamped(v[k][e], scale_at(at));
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

dim3 blocks_of(const Q8Mat &m) { return dim3((m.cols + 127) / 128, (m.rows + 127) / 128); }

// Rows a thread: two, 16 waves a block, where there are fewer than `kTwo` blocks and a
// thread's own time counts; eight, four waves, where there are more.  Along rows 16 waves
// are faster until the CUs are full (256 blocks of bf16 3.6 us for 4.5, 512 4.8 for 5.3,
// 1024 10.1 for 9.4; fp32 alike).  Down columns, the waves' maxima meet in LDS, where 16
// cost four times what four do, and a second block no longer fits beside a first: both ways
// 32 blocks 5.1 for 5.8, 256 6.3 for 6.7, 288 9.5 for 7.2; columns alone 4.5 for 4.4, 5.2
// for 4.9, 7.9 for 5.5.  Of fp32 1,024 threads have not the registers for it as well (both
// ways 32 blocks 14.7 for 6.2, 512 33.0 for 11.4), and eight rows are right throughout.
template <bool kF32, int WHAT>
constexpr unsigned kTwo = WHAT == kWriteRows             ? 1024u
                          : kF32 || WHAT == kWriteCols ? 0u
                                                         : 257u;

template <int FMT, bool kF32, int WHAT>
void quantize(const void *x, int64_t ldx, const Q8Mat &a, const Q8Mat &b, hipStream_t st) {
    const dim3 grid = blocks_of(a);
    if constexpr (kTwo<kF32, WHAT> > 0) {
        if (grid.x * grid.y < kTwo<kF32, WHAT>) {
            q8_quantize_kernel<FMT, kF32, WHAT, 2><<<grid, 1024, 0, st>>>(x, ldx, a, b);
            return;
        }
    }
    q8_quantize_kernel<FMT, kF32, WHAT, 8><<<grid, 256, 0, st>>>(x, ldx, a, b);
}

template <int FMT, bool kF32>
void quantize(const void *x, int64_t ldx, const Q8Mat &a, const Q8Mat *b, hipStream_t st) {
    const Q8Mat none{};
    if (b != nullptr) quantize<FMT, kF32, kWriteRows | kWriteCols>(x, ldx, a, *b, st);
    else if (a.blocks == FSDP_Q8_ROWS) quantize<FMT, kF32, kWriteRows>(x, ldx, a, none, st);
    else if (a.blocks == FSDP_Q8_COLS) quantize<FMT, kF32, kWriteCols>(x, ldx, a, none, st);
    else quantize<FMT, kF32, kWriteTiles>(x, ldx, a, none, st);
}

template <int FMT, bool kF32, bool kDiv>
void dequantize(const Q8Mat &q, void *out, int64_t ldo, hipStream_t st) {
    const dim3 grid = blocks_of(q);
    // as above, nothing meeting in LDS (by columns to bf16, 64 blocks 3.4 us for 4.1, 512 6.3
    // for 6.4, 1024 11.0 for 10.6, 2048 18.4 for 16.9; other blocks and fp32 alike)
    if (grid.x * grid.y < 1024u) q8_dequantize_kernel<FMT, kF32, 2, kDiv><<<grid, 1024, 0, st>>>(q, out, ldo);
    else q8_dequantize_kernel<FMT, kF32, 8, kDiv><<<grid, 256, 0, st>>>(q, out, ldo);
}

template <int FMT, bool kF32>
void dequantize(const Q8Mat &q, void *out, int64_t ldo, hipStream_t st) {
    // (with the division's code in it, unused, 4097 x 1408 takes 8.5 us for 5.9)
    q.divisor ? dequantize<FMT, kF32, true>(q, out, ldo, st)
              : dequantize<FMT, kF32, false>(q, out, ldo, st);
}

}  // namespace

hipError_t launch_q8_quantize(const void *x, bool f32, int64_t ldx, const Q8Mat &a, const Q8Mat *b,
                              hipStream_t st) {
    if (a.rows == 0 || a.cols == 0) return hipSuccess;
    const Q8Mat &rows = b && a.blocks == FSDP_Q8_COLS ? *b : a;
    const Q8Mat *cols = b && a.blocks == FSDP_Q8_COLS ? &a : b;
    if (a.format == FSDP_Q8_E4M3)
        f32 ? quantize<FSDP_Q8_E4M3, true>(x, ldx, rows, cols, st)
            : quantize<FSDP_Q8_E4M3, false>(x, ldx, rows, cols, st);
    else
        f32 ? quantize<FSDP_Q8_E5M2, true>(x, ldx, rows, cols, st)
            : quantize<FSDP_Q8_E5M2, false>(x, ldx, rows, cols, st);
    return hipGetLastError();
}

hipError_t launch_q8_dequantize(const Q8Mat &q, void *out, bool f32, int64_t ldo, hipStream_t st) {
    if (q.rows == 0 || q.cols == 0) return hipSuccess;
    if (q.format == FSDP_Q8_E4M3)
        f32 ? dequantize<FSDP_Q8_E4M3, true>(q, out, ldo, st)
            : dequantize<FSDP_Q8_E4M3, false>(q, out, ldo, st);
    else
        f32 ? dequantize<FSDP_Q8_E5M2, true>(q, out, ldo, st)
            : dequantize<FSDP_Q8_E5M2, false>(q, out, ldo, st);
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
