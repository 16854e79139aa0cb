// How an orthogonalised update runs: the bounds that scale its operands, the
// tiles of its products and how they are dealt, the workspace.  Host code.  Internal
// header.
#pragma once

#include <cmath>

#include "ring_plan.h"

namespace dgor {
namespace newton_schulz {

// The three products of a step.
enum Which { kGram, kPolynomial, kUpdate };

// Elements of a row of two terms of `cols` columns (Pair, orthogonalize.hip).
inline int pair_stride(int cols) { return 2 * ((cols + 31) / 32 * 32); }

constexpr size_t kWsAlign = 256;
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
// A launch holds fewer than 2^32 threads; the products' tiles are dealt to at most
// 256 workgroups, and counted in ints.
constexpr long long kMostGroups = 1 << 24, kMostTiles = 1 << 30;

// How a product runs.
enum Tile { kTile256, kTile128, kTile64 };
constexpr int side_of(Tile t) { return t == kTile256 ? 256 : t == kTile128 ? 128 : 64; }

inline int results_cols(Which which, int m, int n) { return which == kUpdate ? n : m; }

inline long long tiles_of(Which which, int m, int n, Tile t)
{
    const long long down = ceil_div(m, side_of(t));
    return which == kUpdate ? down * ceil_div(n, side_of(t)) : down * (down + 1) / 2;
}

struct Way {
    Tile tile;
    int groups, whole, run;   // of Work
    bool joined;
    size_t slabs;             // bytes
};

// Microseconds of a tile: its ends (with A's part in the polynomial's), and each
// stage, where up to 64 compute units work and where 192 and more do (between them
// in between: 136 tiles of 256 x 256 take 2.0).  Over 102 products (129 to 4096 rows,
// sums of 128 to 8192, batches of 1 to 30) what is chosen is the shortest of the three
// tiles, with and without runs, for 95, at most 1.12 times it for 100, and 1.22 and 1.19
// times for two long sums in few 64 x 64 tiles, which runs do not shorten.
struct TileCost {
    Tile tile;
    double ends, polynomial, few, all;
};
constexpr TileCost kTiles[] = {{kTile256, 16.0, 10.0, 1.58, 2.3}, {kTile128, 7.0, 3.0, 0.58, 0.75},
                               {kTile64, 4.0, 0.5, 0.206, 0.24}};
constexpr int kUnits = 256;                       // compute units
constexpr double kJoin = 5.0, kSlabBytes = 3e6;   // a join's launch; a microsecond's bytes of slabs

// The tile and the way its stages are dealt.
inline bool choose(Which which, int m, int n, int batch, Way &best)
{
    const int stages = ceil_div(which == kGram ? n : m, 32);
    double least = 0;
    bool any = false;
    for (const TileCost &c : kTiles) {
        const long long tiles = batch * tiles_of(which, m, n, c.tile);
        if (tiles >= kMostTiles)
            continue;
        const double ends = c.ends + (which == kPolynomial ? c.polynomial : 0.0);
        const auto stage = [&](long long groups) {
            const double busy = (double)(groups - 64) / 128;
            return c.few + (c.all - c.few) * (busy < 0 ? 0.0 : busy > 1 ? 1.0 : busy);
        };
        const long long rounds = (tiles + kUnits - 1) / kUnits;
        const double whole = rounds * (ends + stages * stage(tiles));
        if (!any || whole < least) {
            any = true, least = whole;
            best = {c.tile, (int)(tiles < kUnits ? tiles : kUnits), (int)tiles, 1, false, 0};
        }
        // whole tiles in full rounds, the rest's stages in runs of at least four
        const long long rest = tiles % kUnits;
        for (int groups : {kUnits, kUnits * 3 / 4, kUnits / 2, kUnits / 4}) {
            const long long run = (rest * stages + groups - 1) / groups;
            if (rest == 0 || run < 4 || run >= stages || (tiles > kUnits && groups < kUnits))
                continue;
            const size_t bytes = (size_t)2 * groups * side_of(c.tile) * side_of(c.tile) * sizeof(float);
            // (a run is of up to two tiles, at an end of each)
            const double us = (double)(tiles / kUnits) * (ends + stages * c.all) + 2.0 * c.ends + run * stage(groups) +
                              kJoin + bytes / kSlabBytes;
            if (us < least) {
                least = us;
                best = {c.tile, groups, (int)(tiles - rest), (int)run, true, bytes};
            }
        }
    }
    return any;
}

// Bounds of a step: of X's singular values, and of the polynomial on X X^T's
// eigenvalues.  |a s + b s^3 + c s^5| and |a + b t + c t^2| over [0, r] and [0,
// r^2]: at the ends and where the derivative is zero.
inline double grown(double a, double b, double c, double r)
{
    const auto f = [&](double s) { return std::fabs(s * (a + s * s * (b + s * s * c))); };
    double most = f(r);
    const auto at = [&](double t) {   // a zero of a + 3 b t + 5 c t^2, t = s^2
        if (t > 0 && t < r * r)
            most = std::fmax(most, f(std::sqrt(t)));
    };
    // (the sum that does not cancel gives one zero and the product of both, a / 5 c, the
    // other: a c that is next to nothing leaves the cubic's)
    const double d = 9 * b * b - 20 * a * c;
    if (d >= 0) {
        const double q = -(3 * b + std::copysign(std::sqrt(d), b)) / 2;
        at(q / (5 * c));   // not a number or infinite where there is none
        at(a / q);
    }
    return most;
}
inline double multiplied(double a, double b, double c, double r)
{
    const double t = r * r;
    const auto f = [&](double v) { return std::fabs(a + v * (b + v * c)); };
    double most = std::fmax(f(0), f(t));
    if (c != 0 && -b / (2 * c) > 0 && -b / (2 * c) < t)
        most = std::fmax(most, f(-b / (2 * c)));
    return most;
}
// What a step's bounds may be: below kLeast an operand would want a power of two whose
// products, undone, leave FP32.
constexpr double kLeast = 0x1p-35, kMost = 256;
inline bool in_range(double bound) { return bound == 0 || (bound >= kLeast && bound <= kMost); }
// The power of two at which values of at most `most` stay binary16: the rounding
// of the sums is far below what 60000 leaves to 65504.
inline int exponent_for(double most)
{
    if (most == 0)
        return 0;
    int e = 0;
    std::frexp(60000.0 / most, &e);   // 60000 / most in [2^(e - 1), 2^e)
    return e - 1;
}

struct Step {
    double a, b, c;
    int x, gram, poly;   // exponents of X, A and P
};

struct Layout {
    bool small;              // all steps in one launch
    int strips, width, mp;   // or, strips > 0, a step in one launch (x[0]: X, gram and poly: A's parts)
    int m, n, ldx, lda;
    bool turned_in, turned_out;
    int blocks, lg;          // of the sums of squares
    Way way[3];
    Step step[GEMM_MAX_STEPS];
    double last;             // `scale`, and the last step's powers of two undone
    size_t sums, x[2], gram, poly, part, bytes;   // offsets, and the whole size
};

// What the small kernel's LDS and registers hold.
constexpr int kSmallWaves = 16, kSmallBytes = 159 * 1024;
constexpr int kSmallUnits = 6;     // units of eight of G a thread loads
constexpr int kSmallBlocks = 10;   // 16 x 16 blocks of X a wavefront computes
// Strips of a matrix of few rows: so many at most, whose parts of A every workgroup
// reads, and a strip's 16-byte units a thread holds.
constexpr int kMostStrips = 8, kStripUnits = 8;
// Which of the two, or the three products a step, by five steps in FP32, measured in
// us as all steps in one launch / strips / products.  Up to kSmallStages of a
// wavefront's 32-deep block products a step, one launch: 64 x 64 (6) 29 / 33 / 77,
// 64 x 128 (10) 35 / 35.  Past it strips, 64 x 256 (18) 50 / 36, 32 x 1024 (41)
// 71 / 35, 128 x 128 68 with strips and 91 without, 16 x 3000 41 and 174, where they
// are one workgroup a compute unit; else again one launch where a matrix fits it: 64
// of 64 x 512 83 / 109, 600 of 96 x 200 226 / 525 / 545.  What does not: strips up to
// two workgroups a compute unit (64 of 64 x 800 129 and 167, 64 of 128 x 256 109 and
// 129; 200 of each 341 and 295, 354 and 269), any number of up to 32 rows, of
// which the products' tiles would be half empty (600 of 16 x 3000 840 and 1502).
constexpr int kSmallStages = 16;
inline long long small_stages(int m, int n)
{
    const int mb = ceil_div(m, 16), nb = ceil_div(n, 16), mt = ceil_div(m, 32), nt = ceil_div(n, 32);
    return (long long)ceil_div(mb * mb, kSmallWaves) * (nt + mt) + (long long)ceil_div(mb * nb, kSmallWaves) * mt;
}

inline bool ld_ok(int ld, int row) { return ld >= (row > 1 ? row : 1); }

// Whether two of a stack's results share an element.  Matrices may lie between each
// other's rows: one that begins d further has a row that begins d % ld into one of the
// first's, as long as d is inside it.
inline bool results_overlap(const gemm_orthogonalize_params &q)
{
    const long long rows = q.op_o ? q.N : q.M, cols = q.op_o ? q.M : q.N, ld = q.ldo;
    if (q.batch <= 1 || rows == 0 || cols == 0)
        return false;
    if (q.stride_o < -(1LL << 62) || q.stride_o > (1LL << 62))
        return true;   // past every address: the sums below would overflow
    const long long by = q.stride_o < 0 ? -q.stride_o : q.stride_o;
    if (by >= cols && by <= ld && (q.batch - 1) * by + cols <= ld)   // all in one row's stride
        return false;
    for (long long i = 1, d = by; i < q.batch && d < (rows - 1) * ld + cols; ++i, d += by) {
        const long long row = d / ld, in = d - row * ld;
        if (in < cols || (row + 1 < rows && ld - in < cols))
            return true;
    }
    return false;
}

inline int lay_out(const gemm_orthogonalize_params *q, Layout &l)
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    constexpr int LONGEST = (1 << 21) - 32;   // offsets in a tile's 256 rows stay below 2^31 bytes
    if (q->batch < 0 || q->M < 0 || q->N < 0 || q->M > LONGEST || q->N > LONGEST || q->steps < 1 ||
        q->steps > GEMM_MAX_STEPS || !(q->eps >= 0))
        return GEMM_ERR_INVALID_DIM;
    if ((q->op_g != GEMM_OP_N && q->op_g != GEMM_OP_T) || (q->op_o != GEMM_OP_N && q->op_o != GEMM_OP_T) ||
        !ld_ok(q->ldg, q->op_g ? q->M : q->N) || !ld_ok(q->ldo, q->op_o ? q->M : q->N))
        return GEMM_ERR_INVALID_LAYOUT;
    l = Layout{};
    double r = 1;
    for (int i = 0; i < q->steps; ++i) {
        Step &s = l.step[i];
        s.a = q->coefficients[3 * i], s.b = q->coefficients[3 * i + 1], s.c = q->coefficients[3 * i + 2];
        if (!std::isfinite(s.a) || !std::isfinite(s.b) || !std::isfinite(s.c))
            return GEMM_ERR_INVALID_COEFFICIENTS;
        const double p = multiplied(s.a, s.b, s.c, r), next = grown(s.a, s.b, s.c, r);
        if (!in_range(p) || !in_range(next))
            return GEMM_ERR_INVALID_COEFFICIENTS;
        s.x = exponent_for(r), s.gram = exponent_for(r * r), s.poly = exponent_for(p);
        r = next;
    }
    // what the last sums are multiplied by, a normal FP32 number
    const Step &end = l.step[q->steps - 1];
    l.last = std::ldexp(q->scale, -end.poly - end.x);
    if (std::isfinite(q->scale) && q->scale != 0 && !(std::fabs(l.last) >= 0x1p-126 && std::fabs(l.last) < 0x1p127))
        return GEMM_ERR_INVALID_COEFFICIENTS;
    if (q->batch == 0 || q->M == 0 || q->N == 0)
        return GEMM_OK;
    const bool tall = q->M > q->N;
    l.m = tall ? q->N : q->M, l.n = tall ? q->M : q->N;
    l.turned_in = tall != (q->op_g == GEMM_OP_T), l.turned_out = tall != (q->op_o == GEMM_OP_T);
    // Strips: LDS holds one and A, the registers its units and its 16 x 16 blocks.
    const long long mp = (l.m + 31LL) / 32 * 32, np = (l.n + 31LL) / 32 * 32;
    const int mb = ceil_div(l.m, 16);
    l.mp = (int)mp;
    l.width = (int)std::fmax(64.0, (l.n + 32LL * kMostStrips - 1) / (32LL * kMostStrips) * 32LL);
    const long long groups = (long long)q->batch * ceil_div(l.n, l.width);
    const bool strips = mp <= 128 && 4 * mp * (mp + l.width) <= kSmallBytes &&
                        4 * mp * l.width <= 16 * 64 * kSmallWaves * kStripUnits &&
                        (long long)mb * (l.width / 16) <= kSmallWaves * kSmallBlocks && groups < kMostGroups / 4;
    // One launch: LDS holds X and A, the registers 16 x 16 blocks and G's units.
    const int cols = l.turned_in ? l.m : l.n, rows = l.turned_in ? l.n : l.m;
    l.small = mp <= 128 && 4 * mp * (mp + np) <= kSmallBytes &&
              mb * ceil_div(l.n, 16) <= kSmallWaves * kSmallBlocks &&
              (long long)rows * ceil_div(cols, 8) <= 64 * kSmallWaves * kSmallUnits && q->batch < kMostGroups / 4 &&
              (!strips || small_stages(l.m, l.n) <= kSmallStages || groups > kUnits);
    if (l.small)
        return GEMM_OK;
    const auto take = [&](size_t bytes) {
        const size_t at = l.bytes;
        l.bytes += round_up(bytes, kWsAlign);
        return at;
    };
    if (strips && (groups <= 2 * kUnits || mp == 32)) {
        l.strips = ceil_div(l.n, l.width);
        l.x[0] = take((size_t)groups * 4 * l.mp * l.width);
        l.gram = take((size_t)groups * mb * (mb + 1) / 2 * 1024);
        l.poly = q->steps > 1 ? take((size_t)groups * mb * (mb + 1) / 2 * 1024) : l.gram;
        return GEMM_OK;
    }
    l.ldx = pair_stride(l.n), l.lda = pair_stride(l.m);
    for (int i = 0; i < 3; ++i)
        if (!choose((Which)i, l.m, l.n, q->batch, l.way[i]))
            return GEMM_ERR_INVALID_DIM;
    if (q->batch * (long long)ceil_div(l.m, 64) * ceil_div(l.n, 64) >= kMostGroups)
        return GEMM_ERR_INVALID_DIM;
    // parts of at least 2048 elements, a unit of eight a thread; at most 1024, four
    // a thread of start_kernel
    const long long parts = ((long long)l.m * l.n + 2047) / 2048;
    l.blocks = (int)(parts < 1024 ? parts : 1024);
    if (q->batch * (long long)l.blocks >= kMostGroups)
        return GEMM_ERR_INVALID_DIM;
    while (l.lg < 8 && (8 << l.lg) < cols)
        ++l.lg;
    const size_t b = (size_t)q->batch, x = 2 * b * l.m * l.ldx, a = 2 * b * l.m * l.lda;
    l.sums = take(sizeof(double) * b * l.blocks);
    l.x[0] = take(x);
    l.x[1] = q->steps > 1 ? take(x) : l.x[0];
    l.gram = take(a);
    l.poly = take(a);
    size_t part = 0;
    for (const Way &w : l.way)
        part = w.slabs > part ? w.slabs : part;
    l.part = take(part);
    return GEMM_OK;
}

}  // namespace newton_schulz
}  // namespace dgor
