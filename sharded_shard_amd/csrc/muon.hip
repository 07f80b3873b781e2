// Muon on the fp32 shards, in one pass each:
//
//   momentum   m = mu*m + (1-mu)*g;  u = nesterov ? mu*m + (1-mu)*g : m
//              and bf16(u) into the rank's all-gather segment
//   update     p = p*(1 - lr*wd) - (lr*s)*o
//              and bf16(p) into the segment, o the bf16 orthogonalised update
//
// Per element each operation is one fp32 rounding, in that order, as for
// AdamW, so that the results do not depend on which kernel ran or how a shard
// is aligned.  The gradient comes from the grad shards or as the mean of the N
// rows of the reduce-scatter input, summed as the reduction does.
//
// All three move 12 to 14 bytes an element (2N + 10 with the reduction) for a
// handful of operations: HBM bounds them.  One decoder block's matrices at 8
// ranks (27 million elements a rank): momentum 64 us, 6.7 TB/s; with the
// reduction 122 us, 6.5; update 55 us, 6.6.  Non-temporal loads and stores of the
// shards are worth a fifth (78 us without either), plain stores of the segment
// 5% over non-temporal ones.  Reserving LDS to hold fewer blocks a CU, which the
// fused AdamW step gains from, costs 3 to 14% here.
#include "muon.hpp"
#include "rows.hpp"

// Cache policy of the shards (bit 0: non-temporal loads, bit 1: stores).
#ifndef FSDP_MUON_POL
#define FSDP_MUON_POL 3
#endif
// the segment is read next by the all-gather: plain stores
#ifndef FSDP_MUON_OUT_NT
#define FSDP_MUON_OUT_NT 0
#endif
// elements per block where one row or none is read (1024 and 4096: 2 and 3%
// slower)
#ifndef FSDP_MUON_SUB
#define FSDP_MUON_SUB 2048
#endif

namespace fsdp {

namespace {

template <bool kNesterov>
struct Momentum {
    float mu, omm;
    __device__ __forceinline__ float operator()(float &m, float g) const {
        const float h = omm * g;
        m = mu * m + h;
        return kNesterov ? mu * m + h : m;
    }
};

struct Update {
    float decay, step;
    __device__ __forceinline__ float operator()(float &p, float o) const {
        p = p * decay - step * o;
        return p;
    }
};

// Store 4 bf16 at p, whose address modulo 8 is k (even, uniform).
__device__ __forceinline__ void store_quad(uint16_t *p, uint32_t k, u32x2 w) {
    if (k == 0) {
        stp<FSDP_MUON_OUT_NT>(reinterpret_cast<u32x2 *>(p), w);
    } else if (k == 4) {
        uint32_t *d = reinterpret_cast<uint32_t *>(p);
        d[0] = w.x;
        d[1] = w.y;
    } else {
        p[0] = static_cast<uint16_t>(w.x);
        *reinterpret_cast<uint32_t *>(p + 1) = alignbyte2(w.y, w.x);
        p[3] = static_cast<uint16_t>(w.y >> 16);
    }
}

// Where a run's inputs come from: the N rows of a bf16 buffer (their mean; N
// = 1 is one row as it is), or fp32 shards.
struct Rows {
    const uint16_t *row0;
    int64_t S;
    int32_t N;
    float fN;
    __device__ __forceinline__ float mean(float x) const { return N == 1 ? x : x / fN; }
    __device__ __forceinline__ float at(int64_t e) const {
        return mean(sum_rows_scalar(row0, S, N, e));
    }
};
struct Grad {
    const float *g;
    __device__ __forceinline__ float at(int64_t e) const { return g[e]; }
};

template <class Op, class Src>
__device__ __forceinline__ void scalar_at(float *X, const Src &src, uint16_t *dst, int64_t e,
                                          const Op &op) {
    float x = X[e];
    const float y = op(x, src.at(e));
    X[e] = x;
    if (dst != nullptr) dst[e] = static_cast<uint16_t>(bf16_rne(y));
}

// Valid elements [0, valid) of one run of the state X, its outputs into dst
// (null: none), zeros in dst from valid to len.  A quad per lane and pass, two
// passes in flight: every load and store instruction of a wave is contiguous
// (rows 512 bytes, the state 1 KB, the bf16 output 512 bytes), through buffer
// ranges of the run, so that all loads leave before the first wait and lanes
// past the end need no branch.  kAl: the rows' quads are 8-byte aligned; else
// each row is funnel-shifted by its own phase.
template <class Op, class Src, int RB, bool kAl>
__device__ __forceinline__ void muon_run(float *X, const Src &src, uint16_t *dst, int64_t len,
                                         int64_t valid, const Op &op) {
    constexpr int LN = FSDP_MUON_POL & 1, SN = (FSDP_MUON_POL >> 1) & 1, QP = 2;
    constexpr bool kRows = __is_same(Src, Rows);
    const int tid = threadIdx.x;
    const uint32_t ap = lo32(X) & 15u;
    int64_t head = ((16u - ap) & 15u) >> 2;
    if (head > valid) head = valid;
    // the state and the fp32 source take the same 16-byte phase, aligned rows
    // their own 8-byte one; what does not fit goes element by element
    bool vec = true;
    uint32_t k0 = 0, kS = 0;
    if constexpr (kRows) {
        k0 = lo32(src.row0 + head) & 7u;
        kS = static_cast<uint32_t>((src.S * 2) & 7);
        vec = !kAl || (k0 | kS) == 0;
    } else {
        vec = ap == (lo32(src.g) & 15u);
    }
    if (!vec) {
        for (int64_t e = tid; e < valid; e += blockDim.x) scalar_at(X, src, dst, e, op);
    } else {
        if (tid < head) scalar_at(X, src, dst, tid, op);
        const int64_t nq = (valid - head) >> 2;
        const uint32_t k8 = lo32(dst + head) & 7u;
        const int64_t lane = tid & 63;
        char *xb = reinterpret_cast<char *>(X + head);
        const uint32_t sb = static_cast<uint32_t>(nq) << 4;
        for (int64_t qb = (tid >> 6) * 64 * QP; qb < nq; qb += (blockDim.x >> 6) * 64 * QP) {
            float in[QP][4];
            f32x4 x[QP], g[QP];
#pragma unroll
            for (int h = 0; h < QP; ++h) {
                const uint32_t o = static_cast<uint32_t>(qb + lane + 64 * h) << 4;
                x[h] = __builtin_bit_cast(f32x4, bload16<LN>(xb, o, sb));
                if constexpr (!kRows)
                    g[h] = __builtin_bit_cast(
                        f32x4, bload16<LN>(reinterpret_cast<const char *>(src.g + head), o, sb));
            }
            if constexpr (kRows) {
                const uint32_t dbytes = static_cast<uint32_t>(2 * (valid - head));
                const uint32_t offb = static_cast<uint32_t>(qb + lane) << 3;
                if constexpr (kAl)
                    sum_rows_quad<1, RB, QP>(src.row0 + head, offb, dbytes, src.S, src.N, in);
                else
                    sum_rows_quad_mis<1, RB>(src.row0 + head, offb, dbytes, src.S, src.N, k0, kS,
                                             in);
            }
#pragma unroll
            for (int h = 0; h < QP; ++h) {
                const int64_t q = qb + lane + 64 * h;
                float xe[4] = {x[h].x, x[h].y, x[h].z, x[h].w}, y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if constexpr (kRows) y[k] = op(xe[k], src.mean(in[h][k]));
                    else y[k] = op(xe[k], g[h][k]);
                }
                bstore16<SN>(xb, static_cast<uint32_t>(q) << 4, sb,
                             __builtin_bit_cast(u32x4, f32x4{xe[0], xe[1], xe[2], xe[3]}));
                if (dst != nullptr && q < nq)
                    store_quad(dst + head + (q << 2), k8,
                               u32x2{pack2(y[0], y[1]), pack2(y[2], y[3])});
            }
        }
        const int64_t done = head + (nq << 2);
        if (tid < valid - done) scalar_at(X, src, dst, done + tid, op);
    }
    if (dst != nullptr) zero_bf16<FSDP_MUON_OUT_NT>(dst, valid, len);
}

// Calls f(tile, first element, length, valid elements) for each sub-range of
// this block.
template <class F>
__device__ __forceinline__ void for_tiles(const PackTile *__restrict__ tiles, int64_t n_tiles,
                                          int32_t split, int64_t sub, F &&f) {
    const int64_t nvt = n_tiles * split;
    for (int64_t vt = first_vt(); vt < nvt; vt += gridDim.x) {
        int64_t t, b;
        sub_range(vt, split, sub, &t, &b);
        const PackTile tl = tiles[t];
        if (b >= tl.len) continue;
        const int64_t len = tl.len - b < sub ? tl.len - b : sub;
        int64_t valid = tl.valid - b;
        valid = valid < 0 ? 0 : (valid > len ? len : valid);
        f(tl, b, len, valid);
    }
}

template <bool kNesterov>
__global__ __launch_bounds__(kBlock) void muon_momentum_kernel(
    const PackTile *__restrict__ tiles, int64_t n_tiles, int32_t split, int64_t sub,
    const DevEntry *__restrict__ ents, uint16_t *__restrict__ ag_in, Momentum<kNesterov> op) {
    for_tiles(tiles, n_tiles, split, sub,
              [&](const PackTile &tl, int64_t b, int64_t len, int64_t valid) {
                  const DevEntry en = ents[tl.entry];
                  const int64_t o = tl.src + b;
                  muon_run<Momentum<kNesterov>, Grad, 1, true>(
                      en.exp_avg + o, Grad{en.grad + o}, ag_in + tl.dst + b, len, valid, op);
              });
}

template <bool kNesterov, int RB, bool kAl>
__global__ __launch_bounds__(kBlock) void muon_reduce_momentum_kernel(
    const PackTile *__restrict__ tiles, int64_t n_tiles, int32_t split, int64_t sub,
    const DevEntry *__restrict__ ents, const uint16_t *__restrict__ rs_in,
    uint16_t *__restrict__ ag_in, int64_t S, int32_t N, float fN, Momentum<kNesterov> op) {
    for_tiles(tiles, n_tiles, split, sub,
              [&](const PackTile &tl, int64_t b, int64_t len, int64_t valid) {
                  const DevEntry en = ents[tl.entry];
                  muon_run<Momentum<kNesterov>, Rows, RB, kAl>(
                      en.exp_avg + tl.src + b, Rows{rs_in + tl.dst + b, S, N, fN},
                      ag_in + tl.dst + b, len, valid, op);
              });
}

// The update's source can sit at any even phase against the state's (a full
// tensor's row starts where its columns put it), so the funnel-shifted read of
// one row serves all.
__global__ __launch_bounds__(kBlock) void muon_update_kernel(
    const PackTile *__restrict__ tiles, int64_t n_tiles, int32_t split, int64_t sub,
    const DevEntry *__restrict__ ents, const int64_t *__restrict__ own,
    const uint16_t *__restrict__ upd, uint16_t *__restrict__ ag_in,
    const float *__restrict__ scales, float decay, float lr) {
    for_tiles(tiles, n_tiles, split, sub,
              [&](const PackTile &tl, int64_t b, int64_t len, int64_t valid) {
                  const DevEntry en = ents[tl.entry];
                  const int64_t o = tl.src + b;
                  const uint16_t *src =
                      upd != nullptr ? upd + tl.dst + b : en.full + own[tl.entry] + o;
                  const Update op{decay, scales != nullptr ? lr * scales[tl.entry] : lr};
                  muon_run<Update, Rows, 1, false>(
                      en.master + o, Rows{src, 0, 1, 1.0f},
                      ag_in != nullptr ? ag_in + tl.dst + b : nullptr, len, valid, op);
              });
}

template <bool kNesterov>
void reduce_momentum(hipStream_t st, const PackTile *tiles, int64_t n, const DevEntry *ents,
                     const uint16_t *rs_in, uint16_t *ag_in, int64_t S, int32_t N,
                     const float scal[2], bool aligned) {
    const Momentum<kNesterov> op{scal[0], scal[1]};
    const float fN = static_cast<float>(N);
    auto go = [&](auto kernel, int64_t want, int threads) {
        const int32_t sp = split_for(kTilePack, want);
        kernel<<<grid_for(n, sp), threads, 0, st>>>(tiles, n, sp, kTilePack / sp, ents, rs_in, ag_in,
                                                   S, N, fN, op);
    };
    // Rows in flight and elements a block, from a sweep over both for 1 to 64
    // ranks.  From 16 ranks a wave a block, two rows at a time: 64 ranks 6.4 TB/s
    // (5.95 with four rows, 4.5 with one row and 2048 elements for four waves);
    // misaligned 4.5 (3.9).  Below, three rows at a time where three divide N,
    // else four from four ranks on, the N mod 4 that are left one by one, in fewer
    // elements the more ranks there are: 8 ranks 5.9 TB/s (5.4 with one row and 2048
    // elements), 6 ranks 5.95 (5.45); misaligned rows two at a time, 5.3 TB/s at 6
    // ranks (5.0 with one, 5.1 with three).
    const int64_t most = 6144 / N;
    const int64_t want = most > 2048 ? 2048 : (most < 512 ? 512 : most);
    if (aligned && N >= 16)
        go(muon_reduce_momentum_kernel<kNesterov, 2, true>, 512, 64);
    else if (aligned && N % 3 == 0)
        go(muon_reduce_momentum_kernel<kNesterov, 3, true>, want, kBlock);
    else if (aligned && N >= 4)
        go(muon_reduce_momentum_kernel<kNesterov, 4, true>, want, kBlock);
    else if (aligned)
        go(muon_reduce_momentum_kernel<kNesterov, 2, true>, want, kBlock);
    else if (N >= 16)
        go(muon_reduce_momentum_kernel<kNesterov, 2, false>, 512, 64);
    else
        go(muon_reduce_momentum_kernel<kNesterov, 2, false>, 2048, kBlock);
}

}  // namespace

hipError_t launch_muon_momentum(const PackTile *tiles, int64_t n, const DevEntry *ents,
                                uint16_t *ag_in, const float scal[2], bool nesterov,
                                hipStream_t st) {
    if (n == 0) return hipSuccess;
    const int32_t sp = split_for(kTilePack, FSDP_MUON_SUB);
    const int64_t sub = kTilePack / sp;
    if (nesterov)
        muon_momentum_kernel<true><<<grid_for(n, sp), kBlock, 0, st>>>(
            tiles, n, sp, sub, ents, ag_in, Momentum<true>{scal[0], scal[1]});
    else
        muon_momentum_kernel<false><<<grid_for(n, sp), kBlock, 0, st>>>(
            tiles, n, sp, sub, ents, ag_in, Momentum<false>{scal[0], scal[1]});
    return hipGetLastError();
}

hipError_t launch_muon_reduce_momentum(const PackTile *tiles, int64_t n, const DevEntry *ents,
                                       const uint16_t *rs_in, uint16_t *ag_in, int64_t S,
                                       int32_t N, const float scal[2], bool nesterov,
                                       bool chunk_aligned, hipStream_t st) {
    if (n == 0) return hipSuccess;
    if (nesterov)
        reduce_momentum<true>(st, tiles, n, ents, rs_in, ag_in, S, N, scal, chunk_aligned);
    else
        reduce_momentum<false>(st, tiles, n, ents, rs_in, ag_in, S, N, scal, chunk_aligned);
    return hipGetLastError();
}

hipError_t launch_muon_update(const PackTile *tiles, int64_t n, const DevEntry *ents,
                              const int64_t *own, const uint16_t *upd, uint16_t *ag_in,
                              const float *scales, const float scal[2], hipStream_t st) {
    if (n == 0) return hipSuccess;
    const int32_t sp = split_for(kTilePack, FSDP_MUON_SUB);
    muon_update_kernel<<<grid_for(n, sp), kBlock, 0, st>>>(tiles, n, sp, kTilePack / sp, ents, own,
                                                          upd, ag_in, scales, scal[0], scal[1]);
    return hipGetLastError();
}

}  // namespace fsdp
