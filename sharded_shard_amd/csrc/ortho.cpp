// Orthogonalisation plans: layout of the workspace, work tiles, argument
// checks and the launches of an execution.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>
#include <vector>

#include "../../include/fsdp_shard.h"
#include "ortho.hpp"
#include "state.hpp"

struct fsdp_ortho_plan {
    std::vector<fsdp::OrthoMat> mats;       // matrices with elements; in, out set by bind
    std::vector<int32_t> index;             // their places in the caller's list
    std::vector<fsdp::OrthoCoef> coef;
    std::vector<fsdp::OrthoTile> norm, init, gram, join, poly, apply;
    std::vector<fsdp::OrthoTile> one[3], slabs[3], sums;    // few rows: 32, 64, 128
    int32_t t_gram = 128, t_poly = 128, t_apply = 128, split = 1;   // tiles' sides, parts of X X^T
    bool fine = false;                      // both parts of every operand above 128 rows too
    int32_t n_mats = 0, growth = 0;
    double eps = 0.0;
    int64_t ws_bytes = 0;
    bool bound = false;
    bool f32 = false, typed = false;        // inputs' dtype, set by the first bind
    int device = -1;
    char *dmem = nullptr;                   // mats, then the tile tables
    std::vector<std::pair<uintptr_t, uintptr_t>> spans;  // bytes of the bound matrices
};

namespace {

using fsdp::set_error;

// Singular values that the scaled fp16 products hold: X within 4, B within 16.
constexpr double kMaxSigma = 4.0, kMaxB = 16.0;
constexpr int64_t kMaxSide = 1 << 20, kMaxMin = 1 << 16;

int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Largest |f| of f(s) = a s + b s^3 + c s^5 over [0, top], of |b s^2 + c s^4|,
// and of |f(s) / s|, from the ends and the places where a derivative is 0.
void extremes(double a, double b, double c, double top, double *f, double *g, double *q) {
    std::vector<double> t = {0.0, top * top};      // values of s^2
    if (c != 0.0) t.push_back(-b / (2.0 * c));
    // a + 3 b t + 5 c t^2 = 0: the root of the sum without cancellation, and the
    // other from their product a / (5 c), which is right for a vanishing c too
    const double d = 9.0 * b * b - 20.0 * a * c;
    if (d >= 0.0) {
        const double r = -0.5 * (3.0 * b + std::copysign(std::sqrt(d), b));
        if (c != 0.0) t.push_back(r / (5.0 * c));
        if (r != 0.0) t.push_back(a / r);
    }
    *f = *g = *q = 0.0;
    for (double s2 : t) {
        if (!(s2 >= 0.0 && s2 <= top * top)) continue;
        const double r = a + s2 * (b + s2 * c);
        *f = std::max(*f, std::fabs(std::sqrt(s2) * r));
        *g = std::max(*g, std::fabs(s2 * (b + s2 * c)));
        *q = std::max(*q, std::fabs(r));
    }
}

// Every step is held to the range with singular values of 2% more than the steps
// before it can give, for what the products round.  That room is not handed on:
// 2% a step would add up, and a steep step multiplies it.
constexpr double kSpare = 1.02;

fsdp_status check_coeffs(const double *coeffs, int32_t n_steps, fsdp_ortho_plan *p) {
    double top = 1.0, growth = 0.0;
    for (int32_t k = 0; k < n_steps; ++k) {
        const double a = coeffs[3 * k], b = coeffs[3 * k + 1], c = coeffs[3 * k + 2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c))
            return set_error(FSDP_E_INVAL, "fsdp_ortho_plan_create: coefficient of step " +
                                               std::to_string(k) + " is not finite");
        double f, g, q, f0, g0, q0;
        extremes(a, b, c, top * kSpare, &f, &g, &q);
        if (!(f <= kMaxSigma) || !(g <= kMaxB))
            return set_error(FSDP_E_UNSUPPORTED,
                             "fsdp_ortho_plan_create: the coefficients of step " +
                                 std::to_string(k) +
                                 " take a singular value past 4 or b s^2 + c s^4 past 16");
        extremes(a, b, c, top, &f0, &g0, &q0);
        top = f0;
        growth += std::max(0.0, std::log2(std::max(q, 1e-30)));
        p->coef.push_back({static_cast<float>(a), static_cast<float>(b), static_cast<float>(c)});
    }
    p->growth = static_cast<int32_t>(std::ceil(std::min(growth, 1000.0)));
    return FSDP_OK;
}

// Tiles of one matrix, kBlockA x kBlockB of them at a time, so that tiles that
// follow each other share rows of both operands.
constexpr int32_t kBlockA = 4, kBlockB = 8;
void blocks(int32_t mat, int32_t na, int32_t nb, bool lower, std::vector<fsdp::OrthoTile> *out) {
    for (int32_t b0 = 0; b0 < nb; b0 += kBlockB)
        for (int32_t a0 = 0; a0 < na; a0 += kBlockA)
            for (int32_t b = b0; b < std::min(b0 + kBlockB, nb); ++b)
                for (int32_t a = a0; a < std::min(a0 + kBlockA, na); ++a)
                    if (!lower || b <= a) out->push_back({mat, a, b, 0});
}

// Workgroups go to the GPU's 8 XCDs in turn and each XCD has an L2 of its own:
// of every kXcds * kRun tiles in order, each XCD gets kRun that follow each other.
constexpr size_t kXcds = 8, kRun = 32;
void spread(std::vector<fsdp::OrthoTile> *tiles) {
    const std::vector<fsdp::OrthoTile> in = *tiles;
    size_t done = 0;
    while (done < in.size()) {
        const size_t n = std::min(in.size() - done, kXcds * kRun);
        size_t from = 0;
        for (size_t x = 0; x < kXcds; ++x)
            for (size_t k = x; k < n; k += kXcds) (*tiles)[done + k] = in[done + from++];
        done += n;
    }
}

// Bytes of parts of A that a block sums by itself: more with few matrices, whose
// blocks wait for a launch less, fewer with many, whose blocks all read them
// (64 x 4096, 192 and 384 KB: one matrix 76 and 69 us, 8 87 and 82, 16 103 and 150).
int64_t sums_in_block(const fsdp_ortho_plan &p) {
    int32_t few = 0;
    for (const fsdp::OrthoMat &M : p.mats) few += M.m <= fsdp::kSmallMax;
    return few <= 8 ? 384 << 10 : 192 << 10;
}

// Tile sides and the parts of X X^T's sum: what a model of a launch's time says,
// in clocks.  A CU takes `per` clocks for each element of a tile's sum, and a
// tile no less than `alone` however many CUs are idle; measured on products of
// 256 to 4096 rows (256: 46 clocks where every CU has a tile; 192: 34; 128: 13 each
// and 16 alone; 64: 6 and 11).  Larger tiles read their operands less often, smaller
// ones fill the CUs where there are few: one 4096 x 4096 matrix's a X + B X takes
// 150 us in 256 x 256 tiles and 165 in 128 x 128, one 2048 x 2048's 31 and 12; two
// such matrices' X X^T (272 tiles of 256) 135 and 105.  A split sum costs a launch
// and its fp32 parts' way through memory: X X^T of two 1024 x 8192 matrices takes
// 131 us whole in 128 x 128 tiles, 113 in two parts.
struct Tile {
    int32_t side;
    double per, alone;
};
constexpr Tile kTiles[] = {{256, 46.0, 46.0}, {192, 34.0, 34.0}, {128, 13.0, 16.0}, {64, 6.0, 11.0}};
constexpr double kCus = 256.0, kJoinClocks = 12000.0, kPartBytesPerClock = 2000.0;

enum Product { kXXT, kAA, kBX };

// Clocks of one launch over the plan's matrices.
double clocks(const fsdp_ortho_plan &p, Product what, const Tile &tile, int32_t split) {
    double work = 0.0, shortest = 1e300, longest = 0.0, tiles = 0.0;
    for (const fsdp::OrthoMat &M : p.mats) {
        if (M.m <= fsdp::kSmallMax) continue;
        const double a = (M.mp + tile.side - 1) / tile.side, b = (M.np + tile.side - 1) / tile.side;
        const double n = what == kBX ? a * b : a * (a + 1) / 2;
        const double sum = (p.fine ? 3.0 : 1.0) * (what == kXXT ? M.np : M.mp) / split;
        work += n * split * sum;
        tiles += n;
        shortest = std::min(shortest, sum);
        longest = std::max(longest, sum);
    }
    // whole tiles a CU
    const double busy = std::ceil(work / (kCus * shortest)) * shortest * tile.per;
    const double join = split == 1 ? 0.0
                                   : kJoinClocks + 2.0 * tiles * split * tile.side * tile.side * 4.0 /
                                                       kPartBytesPerClock;
    return std::max(busy, longest * tile.alone) + join;
}

void choose(fsdp_ortho_plan *p) {
    int32_t most = 16;
    bool any = false;
    for (const fsdp::OrthoMat &M : p->mats)
        if (M.m > fsdp::kSmallMax) {
            most = std::min(most, M.np / 128);
            any = true;
        }
    if (!any) return;
    double best[3] = {1e300, 1e300, 1e300};
    for (const Tile &tile : kTiles) {
        int32_t *side[3] = {&p->t_gram, &p->t_poly, &p->t_apply};
        for (Product what : {kXXT, kAA, kBX})
            for (int32_t split = 1; split <= (what == kXXT ? most : 1); ++split) {
                const double t = clocks(*p, what, tile, split);
                if (t >= best[what]) continue;
                best[what] = t;
                *side[what] = tile.side;
                if (what == kXXT) p->split = split;
            }
    }
}

// A matrix of few rows: its slabs; true if it needs no norm of its own (one
// slab: the block that works on it takes it).
template <typename F>
bool few_rows(int32_t id, fsdp::OrthoMat *M, int64_t most, fsdp_ortho_plan *p, F &&take) {
    const int cls = M->mp == 32 ? 0 : M->mp == 64 ? 1 : 2;
    const int32_t nb = fsdp::small_slab(M->mp);
    const int64_t part = static_cast<int64_t>(fsdp::small_part(M->mp)) * 16;
    M->slab = nb;
    if (M->n <= nb) {
        p->one[cls].push_back({id, 0, 0, 0});
        return true;
    }
    // shorter slabs as long as every block can sum their parts by itself
    auto count = [&](int32_t slab) { return (M->n + slab - 1) / slab; };
    while (M->slab > 128 && count(round_up(M->slab / 2, 32)) * part <= most)
        M->slab = static_cast<int32_t>(round_up(M->slab / 2, 32));
    const int32_t slabs = count(M->slab);
    M->t[0] = take(static_cast<int64_t>(slabs) * nb * M->mp * 4);
    M->a = take(slabs * part);
    M->b = take(slabs * part);
    for (int32_t s = 0; s < slabs; ++s) p->slabs[cls].push_back({id, s, 0, 0});
    M->n_sums = slabs;
    if (slabs * part > most) {
        M->n_sums = 1;
        for (int32_t t = 0; t < part / 16 / 256; ++t) p->sums.push_back({id, t, slabs, 0});
    }
    return false;
}

void layout(fsdp_ortho_plan *p) {
    int64_t off = 0;
    auto take = [&](int64_t bytes) {
        const int64_t at = off;
        off += round_up(bytes, 256);
        return at;
    };
    const int64_t most = sums_in_block(*p);
    for (size_t i = 0; i < p->mats.size(); ++i) {
        fsdp::OrthoMat &M = p->mats[i];
        const int32_t id = static_cast<int32_t>(i);
        const int64_t total = static_cast<int64_t>(M.rows) * M.cols;
        if (M.m <= fsdp::kSmallMax && few_rows(id, &M, most, p, take)) continue;
        M.n_parts = static_cast<int32_t>(std::max<int64_t>(
            1, std::min<int64_t>(fsdp::kOrthoParts, total / fsdp::kOrthoPartMin)));
        M.parts = take(M.n_parts * 8);
        M.scal = take(sizeof(fsdp::OrthoScal));
        for (int32_t t = 0; t < M.n_parts; ++t) p->norm.push_back({id, t, 0, 0});
        if (M.m <= fsdp::kSmallMax) continue;
        const int64_t x = static_cast<int64_t>(M.np) * M.mp * 2;
        const int64_t s = static_cast<int64_t>(M.mp) * M.mp * 2;
        M.t[0] = take(x);
        M.t[1] = take(x);
        M.lo = take(x);
        M.a = take(s);
        M.b = take(s);
        if (p->fine) {
            M.lo2 = take(x);
            M.al = take(s);
            M.bl = take(s);
        }
        for (int32_t j = 0; j < M.np / 64; j += fsdp::kInitPieces)
            for (int32_t k = 0; k < M.mp / 64; ++k)
                p->init.push_back({id, k, j, std::min(fsdp::kInitPieces, M.np / 64 - j)});
    }
    choose(p);
    // the matrices with the longest sums first, so that short tiles come last
    std::vector<int32_t> order(p->mats.size());
    for (size_t i = 0; i < order.size(); ++i) order[i] = static_cast<int32_t>(i);
    std::stable_sort(order.begin(), order.end(), [&](int32_t x, int32_t y) {
        return p->mats[x].np > p->mats[y].np;
    });
    for (const int32_t id : order) {
        const fsdp::OrthoMat &M = p->mats[id];
        if (M.m <= fsdp::kSmallMax) continue;
        auto count = [](int32_t side, int32_t tile) { return (side + tile - 1) / tile; };
        blocks(id, count(M.mp, p->t_gram), count(M.mp, p->t_gram), true, &p->gram);
        blocks(id, count(M.mp, p->t_poly), count(M.mp, p->t_poly), true, &p->poly);
        blocks(id, count(M.mp, p->t_apply), count(M.np, p->t_apply), false, &p->apply);
    }
    if (p->split > 1) {
        p->join = p->gram;
        p->gram.clear();
        int32_t part = 0;
        for (fsdp::OrthoTile &t : p->join) {
            t.part = part;
            for (int32_t k = 0; k < p->split; ++k) p->gram.push_back({t.mat, t.ti, t.tj, part++});
        }
        const int64_t sums = take(static_cast<int64_t>(part) * p->t_gram * p->t_gram * 4);
        for (fsdp::OrthoMat &M : p->mats) M.sums = sums;
    }
    p->ws_bytes = off;
    spread(&p->gram);
    spread(&p->join);
    spread(&p->poly);
    spread(&p->apply);
}

// A launch has less than 2^32 threads.
bool fits_launches(const fsdp_ortho_plan &p) {
    auto fits = [](const std::vector<fsdp::OrthoTile> &v, int32_t threads) {
        return v.size() * static_cast<uint64_t>(threads) < (uint64_t{1} << 32);
    };
    bool ok = fits(p.norm, 256) && fits(p.init, 256) && fits(p.sums, 256) &&
              fits(p.gram, fsdp::product_threads(p.t_gram)) &&
              fits(p.poly, fsdp::product_threads(p.t_poly)) &&
              fits(p.apply, fsdp::product_threads(p.t_apply));
    for (int c = 0; c < 3; ++c)
        ok = ok && fits(p.one[c], fsdp::small_threads(32 << c)) &&
             fits(p.slabs[c], fsdp::small_threads(32 << c));
    return ok;
}

// The device tables in their order: matrices, coefficients, tiles.
struct Table {
    const void *src;
    size_t bytes;
};
std::vector<Table> tables(const fsdp_ortho_plan &p, const std::vector<fsdp::OrthoMat> &mats) {
    std::vector<Table> t = {{mats.data(), mats.size() * sizeof(fsdp::OrthoMat)},
                            {p.coef.data(), p.coef.size() * sizeof(fsdp::OrthoCoef)}};
    for (const std::vector<fsdp::OrthoTile> *v :
         {&p.norm, &p.init, &p.gram, &p.join, &p.poly, &p.apply, &p.one[0], &p.one[1], &p.one[2],
          &p.slabs[0], &p.slabs[1], &p.slabs[2], &p.sums})
        t.push_back({v->data(), v->size() * sizeof(fsdp::OrthoTile)});
    return t;
}

fsdp_status hip_error(hipError_t e, const char *what) { return fsdp::set_hip_error(e, what); }

}  // namespace

extern "C" {

fsdp_status fsdp_ortho_plan_create(const int64_t *rows, const int64_t *cols, int32_t n_mats,
                                   const double *coeffs, int32_t n_steps, double eps,
                                   fsdp_ortho_plan **out) {
    if (out == nullptr) return set_error(FSDP_E_INVAL, "fsdp_ortho_plan_create: null out");
    *out = nullptr;
    if (n_mats < 0 || (n_mats > 0 && (rows == nullptr || cols == nullptr)))
        return set_error(FSDP_E_INVAL, "fsdp_ortho_plan_create: null rows or cols");
    if (coeffs == nullptr || n_steps < 1)
        return set_error(FSDP_E_INVAL, "fsdp_ortho_plan_create: need coefficients of one step or more");
    if (n_steps > 64)
        return set_error(FSDP_E_UNSUPPORTED, "fsdp_ortho_plan_create: more than 64 steps");
    if (!(eps >= 0.0) || !std::isfinite(eps))
        return set_error(FSDP_E_INVAL, "fsdp_ortho_plan_create: eps must be finite and not negative");
    fsdp_ortho_plan *p = nullptr;
    try {
        p = new fsdp_ortho_plan();
        p->n_mats = n_mats;
        p->eps = eps;
        fsdp_status s = check_coeffs(coeffs, n_steps, p);
        for (int32_t i = 0; s == FSDP_OK && i < n_mats; ++i) {
            const std::string which = "fsdp_ortho_plan_create: matrix " + std::to_string(i);
            if (rows[i] < 0 || cols[i] < 0)
                s = set_error(FSDP_E_INVAL, which + ": negative rows or cols");
            else if (std::max(rows[i], cols[i]) > kMaxSide || std::min(rows[i], cols[i]) > kMaxMin)
                s = set_error(FSDP_E_UNSUPPORTED, which + ": a side is too long");
            if (s != FSDP_OK || rows[i] == 0 || cols[i] == 0) continue;
            fsdp::OrthoMat M{};
            M.rows = static_cast<int32_t>(rows[i]);
            M.cols = static_cast<int32_t>(cols[i]);
            M.wide = M.rows <= M.cols ? 1 : 0;
            M.m = std::min(M.rows, M.cols);
            M.n = std::max(M.rows, M.cols);
            M.mp = M.m <= fsdp::kSmallMax ? fsdp::small_rows_of(M.m)
                                          : static_cast<int32_t>(round_up(M.m, fsdp::kOrthoPad));
            M.np = static_cast<int32_t>(round_up(M.n, fsdp::kOrthoPad));
            p->mats.push_back(M);
            p->index.push_back(i);
        }
        if (s == FSDP_OK) layout(p);
        if (s == FSDP_OK && !fits_launches(*p))
            s = set_error(FSDP_E_UNSUPPORTED, "fsdp_ortho_plan_create: too many tiles for one launch");
        if (s != FSDP_OK) {
            delete p;
            return s;
        }
        *out = p;
        return FSDP_OK;
    } catch (...) {
        delete p;
        return set_error(FSDP_E_NOMEM, "fsdp_ortho_plan_create: host allocation failed");
    }
}

fsdp_status fsdp_ortho_plan_info(const fsdp_ortho_plan *p, int32_t *n_mats,
                                 int64_t *workspace_bytes) {
    if (p == nullptr || n_mats == nullptr || workspace_bytes == nullptr)
        return set_error(FSDP_E_INVAL, "fsdp_ortho_plan_info: null argument");
    *n_mats = p->n_mats;
    *workspace_bytes = p->ws_bytes;
    return FSDP_OK;
}

fsdp_status fsdp_ortho_plan_set_products(fsdp_ortho_plan *p, int32_t products) try {
    const char *call = "fsdp_ortho_plan_set_products";
    if (p == nullptr) return set_error(FSDP_E_INVAL, std::string(call) + ": null plan");
    if (products != FSDP_ORTHO_FP16 && products != FSDP_ORTHO_FP16X2)
        return set_error(FSDP_E_UNSUPPORTED, std::string(call) + ": products must be FP16 or FP16X2");
    if (p->dmem != nullptr)
        return set_error(FSDP_E_STATE, std::string(call) + ": plan already bound");
    fsdp_ortho_plan next;
    next.mats = p->mats;
    next.index = p->index;
    next.coef = p->coef;
    next.n_mats = p->n_mats;
    next.growth = p->growth;
    next.eps = p->eps;
    next.fine = products == FSDP_ORTHO_FP16X2;
    layout(&next);
    if (!fits_launches(next))
        return set_error(FSDP_E_UNSUPPORTED, std::string(call) + ": too many tiles for one launch");
    *p = std::move(next);
    return FSDP_OK;
} catch (...) {
    return set_error(FSDP_E_NOMEM, "fsdp_ortho_plan_set_products: host allocation failed");
}

fsdp_status fsdp_ortho_bind(fsdp_ortho_plan *p, const void *const *in, uint16_t *const *out,
                            int32_t in_dtype, void *stream) try {
    if (p == nullptr || (p->n_mats > 0 && (in == nullptr || out == nullptr)))
        return set_error(FSDP_E_INVAL, "fsdp_ortho_bind: null plan or array");
    if (in_dtype != FSDP_DTYPE_BF16 && in_dtype != FSDP_DTYPE_F32)
        return set_error(FSDP_E_UNSUPPORTED, "fsdp_ortho_bind: in_dtype must be BF16 or F32");
    // Captured executions read addresses from the tables but hold the kernels of
    // the dtype they were captured with: inputs of another size an element would
    // be read past their end.
    if (p->typed && p->f32 != (in_dtype == FSDP_DTYPE_F32))
        return set_error(FSDP_E_STATE, "fsdp_ortho_bind: plan already bound to inputs of another dtype");
    const uintptr_t esize = in_dtype == FSDP_DTYPE_F32 ? 4 : 2;
    struct Span {
        uintptr_t lo, hi;
        bool out;
        int32_t i;
    };
    std::vector<Span> spans;
    std::vector<fsdp::OrthoMat> mats = p->mats;
    for (size_t k = 0; k < mats.size(); ++k) {
        const int32_t i = p->index[k];
        const std::string which = "fsdp_ortho_bind: matrix " + std::to_string(i);
        if (in[i] == nullptr || out[i] == nullptr)
            return set_error(FSDP_E_INVAL, which + ": null pointer");
        const uintptr_t a = reinterpret_cast<uintptr_t>(in[i]);
        const uintptr_t b = reinterpret_cast<uintptr_t>(out[i]);
        if (a % esize != 0 || b % 2 != 0)
            return set_error(FSDP_E_ALIGN, which + ": pointer misaligned for its type");
        const uintptr_t n = static_cast<uintptr_t>(mats[k].rows) * static_cast<uintptr_t>(mats[k].cols);
        spans.push_back({a, a + n * esize, false, i});
        spans.push_back({b, b + n * 2, true, i});
        mats[k].in = in[i];
        mats[k].out = out[i];
        mats[k].low = in_dtype == FSDP_DTYPE_F32 ? 1 : 0;
    }
    std::sort(spans.begin(), spans.end(), [](const Span &x, const Span &y) { return x.lo < y.lo; });
    // an output may share memory with its own input only: pairs that overlap
    // are adjacent in reach of the running end
    for (size_t x = 0; x < spans.size(); ++x)
        for (size_t y = x + 1; y < spans.size() && spans[y].lo < spans[x].hi; ++y)
            if ((spans[x].out || spans[y].out) &&
                !(spans[x].i == spans[y].i && spans[x].out != spans[y].out))
                return set_error(FSDP_E_INVAL,
                                 "fsdp_ortho_bind: output memory of matrix " +
                                     std::to_string(spans[x].out ? spans[x].i : spans[y].i) +
                                     " overlaps matrix " +
                                     std::to_string(spans[x].out ? spans[y].i : spans[x].i));
    std::vector<std::pair<uintptr_t, uintptr_t>> merged;
    for (const Span &sp : spans)
        if (!merged.empty() && sp.lo <= merged.back().second)
            merged.back().second = std::max(merged.back().second, sp.hi);
        else
            merged.emplace_back(sp.lo, sp.hi);

    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_error(e, "fsdp_ortho_bind: hipGetDevice");
    if (p->dmem != nullptr && dev != p->device)
        return set_error(FSDP_E_STATE, "fsdp_ortho_bind: plan already bound on another device");
    const std::vector<Table> tabs = tables(*p, mats);
    if (p->dmem == nullptr) {
        size_t total = 256;
        for (const auto &t : tabs) total += round_up(static_cast<int64_t>(t.bytes), 256);
        void *mem = nullptr;
        if (hipMalloc(&mem, total) != hipSuccess)
            return set_error(FSDP_E_NOMEM, "fsdp_ortho_bind: hipMalloc of device tables failed");
        p->dmem = static_cast<char *>(mem);
        p->device = dev;
    }
    // executions queued on any stream may still read the tables
    e = hipDeviceSynchronize();
    if (e != hipSuccess) return hip_error(e, "fsdp_ortho_bind: hipDeviceSynchronize");
    p->bound = false;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    char *cur = p->dmem;
    for (const auto &t : tabs) {
        if (t.bytes > 0 && e == hipSuccess)
            e = hipMemcpyAsync(cur, t.src, t.bytes, hipMemcpyHostToDevice, st);
        cur += round_up(static_cast<int64_t>(t.bytes), 256);
    }
    if (e == hipSuccess) e = hipStreamSynchronize(st);
    if (e != hipSuccess) return hip_error(e, "fsdp_ortho_bind: upload");
    p->mats = std::move(mats);
    p->spans = std::move(merged);
    p->f32 = in_dtype == FSDP_DTYPE_F32;
    p->typed = true;
    p->bound = true;
    return FSDP_OK;
} catch (...) {
    return set_error(FSDP_E_NOMEM, "fsdp_ortho_bind: host allocation failed");
}

fsdp_status fsdp_ortho_execute(const fsdp_ortho_plan *p, void *workspace, int64_t workspace_bytes,
                               void *stream) try {
    const char *call = "fsdp_ortho_execute";
    if (p == nullptr) return set_error(FSDP_E_INVAL, "fsdp_ortho_execute: null plan");
    if (!p->bound) return set_error(FSDP_E_STATE, "fsdp_ortho_execute: plan not bound");
    if (p->mats.empty()) return FSDP_OK;
    if ((workspace == nullptr && p->ws_bytes > 0) || workspace_bytes < p->ws_bytes)
        return set_error(FSDP_E_INVAL, "fsdp_ortho_execute: the workspace needs " +
                                           std::to_string(p->ws_bytes) + " bytes");
    const uintptr_t w0 = reinterpret_cast<uintptr_t>(workspace);
    if (w0 % 256 != 0)
        return set_error(FSDP_E_ALIGN, "fsdp_ortho_execute: workspace not 256-byte aligned");
    const uintptr_t w1 = w0 + static_cast<uintptr_t>(p->ws_bytes);
    for (const auto &sp : p->spans)
        if (sp.first < w1 && w0 < sp.second)
            return set_error(FSDP_E_INVAL, "fsdp_ortho_execute: workspace overlaps a bound matrix");
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_error(e, "fsdp_ortho_execute: hipGetDevice");
    if (dev != p->device)
        return set_error(FSDP_E_STATE, "fsdp_ortho_execute: current device differs from the bound one");

    const hipStream_t st = static_cast<hipStream_t>(stream);
    const std::vector<Table> tabs = tables(*p, p->mats);
    const char *cur = p->dmem;
    const char *where[15];
    for (size_t t = 0; t < tabs.size(); ++t) {
        where[t] = cur;
        cur += round_up(static_cast<int64_t>(tabs[t].bytes), 256);
    }
    const auto *mats = reinterpret_cast<const fsdp::OrthoMat *>(where[0]);
    const auto *coefs = reinterpret_cast<const fsdp::OrthoCoef *>(where[1]);
    auto tiles = [&](int t) { return reinterpret_cast<const fsdp::OrthoTile *>(where[t]); };
    const fsdp::OrthoTile *norm = tiles(2), *init = tiles(3), *gram = tiles(4), *join = tiles(5),
                          *poly = tiles(6), *apply = tiles(7), *sums = tiles(14);
    auto count = [](const std::vector<fsdp::OrthoTile> &v) { return static_cast<int64_t>(v.size()); };
    const int32_t n_steps = static_cast<int32_t>(p->coef.size());
    const int32_t fine = p->fine ? fsdp::kTileFine : 0;
    auto run = [&](const std::vector<fsdp::OrthoTile> &v, auto &&launch) {
        if (v.empty() || e != hipSuccess) return;
        e = fsdp::injected_fault();
        if (e == hipSuccess) e = launch();
    };
    // matrices of few rows: the classes' one-slab launches, or one of the slabs'
    auto small = [&](int32_t mode, int32_t step) {
        for (int c = 0; c < 3; ++c) {
            const std::vector<fsdp::OrthoTile> &v = mode == fsdp::kSmallAll ? p->one[c] : p->slabs[c];
            run(v, [&] {
                return fsdp::launch_ortho_small(32 << c, tiles((mode == fsdp::kSmallAll ? 8 : 11) + c),
                                                count(v), mats, workspace, p->f32, mode, step,
                                                n_steps, coefs, p->eps, p->growth, st);
            });
        }
    };
    run(p->norm, [&] {
        return fsdp::launch_ortho_norm(norm, static_cast<int64_t>(p->norm.size()), mats, workspace,
                                       p->f32, st);
    });
    small(fsdp::kSmallAll, 0);
    small(fsdp::kSmallStart, 0);
    run(p->init, [&] {
        return fsdp::launch_ortho_init(init, static_cast<int64_t>(p->init.size()), mats, workspace,
                                       p->f32, p->eps, p->growth, st);
    });
    for (size_t k = 0; k < p->coef.size(); ++k) {
        const int32_t src = static_cast<int32_t>(k & 1);
        const bool last = k + 1 == p->coef.size();
        run(p->sums, [&] {
            return fsdp::launch_ortho_sums(sums, count(p->sums), mats, workspace,
                                           static_cast<int32_t>(k), st);
        });
        small(last ? fsdp::kSmallLast : fsdp::kSmallStep, static_cast<int32_t>(k));
        run(p->gram, [&] {
            return fsdp::launch_ortho_gram(p->t_gram | fine, gram, count(p->gram), join, count(p->join),
                                           p->split, mats, workspace, src, k == 0, st);
        });
        run(p->poly, [&] {
            return fsdp::launch_ortho_poly(p->t_poly | fine, poly, count(p->poly), mats, workspace,
                                           p->coef[k], st);
        });
        run(p->apply, [&] {
            return fsdp::launch_ortho_apply(p->t_apply | fine, apply, count(p->apply), mats,
                                            workspace, src, k == 0, k == 0 && !p->f32, last,
                                            p->coef[k], st);
        });
    }
    return e == hipSuccess ? FSDP_OK : hip_error(e, (std::string(call) + ": launch").c_str());
} catch (...) {
    return set_error(FSDP_E_NOMEM, "fsdp_ortho_execute: host allocation failed");
}

void fsdp_ortho_plan_destroy(fsdp_ortho_plan *p) {
    if (p == nullptr) return;
    if (p->dmem != nullptr) {
        int cur = -1;
        (void)hipGetDevice(&cur);
        (void)hipSetDevice(p->device);
        (void)hipDeviceSynchronize();
        (void)hipFree(p->dmem);
        if (cur >= 0) (void)hipSetDevice(cur);
    }
    delete p;
}

}  // extern "C"
