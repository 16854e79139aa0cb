// C entry points of the dense layer and the gated up-projection (declared in
// include/gemm.h): argument checks, choice of kernel, workspace layout.
// Host code only; the kernels live in linear_skinny.hip, linear_ring.hip,
// linear_tile.hip and act_grad.hip.
#include <stdint.h>

#include "linear.h"
#include "ring_plan.h"

namespace {

using dgor::Epilogue;
using dgor::Product;
using dgor::RingCost;
using dgor::RingTimes;
using dgor::ceil_div;
using dgor::kJoinLaunch;
using dgor::kRings;
using dgor::kRingTiles;
using dgor::tiles;

constexpr size_t kWsAlign = 256;
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// A launch holds fewer than 2^32 threads.  With fewer than 2^22 blocks of 128 x
// 64 the smallest tiles, 64 x 32 (gated) or two of 64 x 64 (both weights'
// gradients), are fewer than 2^24 of 256 threads; kernels that would need more
// are not chosen.
constexpr long long kThreads = 1LL << 32;
bool too_large(long long rows, long long cols) { return (rows + 127) / 128 * ((cols + 63) / 64) >= (1LL << 22); }
bool ld_ok(int ld, int row) { return ld >= (row > 1 ? row : 1); }
bool op_ok(int op) { return op == GEMM_OP_N || op == GEMM_OP_T; }
bool act_ok(int act) { return act >= GEMM_ACT_NONE && act <= GEMM_ACT_SILU; }
// The backward passes' activation carries flags.
constexpr int kFlags = GEMM_ROUND_GRADIENT | GEMM_ONLY_F16 | GEMM_ONLY_BF16 | GEMM_NO_INPUT_GRADIENT | GEMM_NO_WEIGHT_GRADIENT;
int act_of(int activation) { return activation & ~kFlags; }
bool wants_input(int activation) { return !(activation & GEMM_NO_INPUT_GRADIENT); }
bool wants_weight(int activation) { return !(activation & GEMM_NO_WEIGHT_GRADIENT); }
bool takes(bool bf16, int activation) { return !(activation & (bf16 ? GEMM_ONLY_F16 : GEMM_ONLY_BF16)); }
bool missing(const void *p, long long rows, long long cols) { return rows > 0 && cols > 0 && !p; }

// How a product runs: the kernel, a ring's tile and, where its tiles leave
// compute units idle, into how many parts the sum over k is split.
enum class Kernel { Rows, Ring, Tile };
struct Way {
    Kernel kernel;
    dgor::RingTile tile;
    int splits, chunk;
    double us;   // the time that a ring was chosen for, or that few rows take
};

// Whether the few-row kernel takes a product.
bool few_rows(const Product &p)
{
    return !p.trans_a && p.nbatch == 1 && p.M <= dgor::kSkinnyRows && dgor::spans_a_unit(p) && !p.opened &&
           512LL * ceil_div(p.N, dgor::skinny_strip(p, false)) < kThreads;
}

// Whether sizes and strides let the rings run (the addresses apart).
bool ring_sizes(const Product &p)
{
    const auto ok = [](int ld) { return ld % 8 == 0 && ld < (1 << 22); };
    return p.units && ok(p.lda) && ok(p.ldb);
}
bool ring_addresses(const Product &p)
{
    const auto all = [](const dgor::Side &s) { return (uintptr_t)s.p | (uintptr_t)s.matrix | (uintptr_t)s.term; };
    return ((all(p.A) | all(p.B)) & 15) == 0;
}

void split(int stages, long long parts, Way &w)
{
    w.splits = 1, w.chunk = 0;
    if (parts > 1) {
        w.chunk = ceil_div(stages, parts);
        w.splits = ceil_div(stages, w.chunk);
    }
}

// Stages of 64 k from which few rows' sums over a K x N matrix are split.  At 40
// whole and split take 9.4 and 8.1 us (1 row, 512 outputs), 14.0 and 11.8 (4096), 17.7
// and 15.1 (48 rows); at 24 6.8 and 8.3, 9.9 and 10.7, 12.7 and 13.1; at 32 they are level.
constexpr int kSplitRows = 40;
// Weights that the few-row kernel reads in a microsecond, past 3 us: 33.5 MB
// 11 us, 134 MB 28 us.
constexpr double kRowsBytes = 5e6;
// The best split of a product on a ring's tile.
Way best_on(const Product &p, const RingCost &c)
{
    Way w{Kernel::Ring, c.tile, 1, 0, 0};
    // parts until two rounds are full, at least two stages of 64 k each
    const int stages = dgor::product_stages(p);
    const long long n = tiles(p, ring_tile_m(c.tile), ring_tile_n(c.tile));
    int best = 1;
    for (int parts : {1, 2, 3, 4, 6, 8, 12, 16}) {
        if (parts > 1 && (2 * parts > stages || n * parts > 512 * c.share))
            break;
        const double t = microseconds(p, c, n, parts);
        if (parts == 1 || t < w.us)
            w.us = t, best = parts;
    }
    split(stages, best, w);
    return w;
}

// The best on each tile, of kRings' order; found once a plan.
struct RingWays {
    Way on[kRingTiles];
};

// `ways`: a product's on the rings, null off them.
Way choose(const Product &p, const RingWays *ways)
{
    Way w{Kernel::Rows, dgor::kRing64, 1, 0, 0};
    if (few_rows(p)) {
        const int stages = dgor::row_stages(p);
        // a K x N matrix with a long sum and too few columns for the compute
        // units: parts of at least eight stages, one for each wavefront
        const long long strips = ceil_div(p.N, dgor::skinny_strip(p, true));
        if (!p.trans_b && stages >= kSplitRows && strips < 256) {
            long long want = (256 + strips - 1) / strips;
            want = want < stages / 8 ? want : stages / 8;
            split(stages, want < 32 ? want : 32, w);
        }
        w.us = 3.0 + 2.0 * (p.nseg / p.terms) * p.K * p.N / kRowsBytes + (w.splits > 1 ? kJoinLaunch : 0.0);
        return w;
    }
    if (ways) {
        for (const Way &v : ways->on)
            if (w.kernel != Kernel::Ring || v.us < w.us)
                w = v;
        return w;
    }
    // the plain tile: split until two workgroups a compute unit, keeping at
    // least four stages a part
    w.kernel = Kernel::Tile;
    const int stages = dgor::product_stages(p);
    const long long n = tiles(p, dgor::kTile, dgor::kTile);
    if (n > 0 && n < 256 && stages >= 8) {
        long long want = 512 / n;
        want = want < stages / 4 ? want : stages / 4;
        split(stages, want < 16 ? want : 16, w);
    }
    return w;
}

// How a product runs off and on the rings, as the operands' addresses will
// have it, and the bytes of its FP32 partial sums either way.
struct Plan {
    Way off, ring;
    size_t part;
};
RingWays ring_ways(const Product &p)
{
    RingWays w;
    for (int i = 0; i < kRingTiles; ++i)
        w.on[i] = best_on(p, kRings[i]);
    return w;
}
Plan plan(const Product &p, const RingWays *ways)   // null: its strides are not the rings'
{
    const auto bytes = [&](const Way &w) {
        return w.splits <= 1 ? 0 : (size_t)(p.gated ? 2 : p.nbatch) * w.splits * dgor::part_size(p) * sizeof(float);
    };
    Plan l;
    l.off = choose(p, nullptr);
    l.ring = ways ? choose(p, ways) : l.off;
    l.part = round_up(bytes(l.off) > bytes(l.ring) ? bytes(l.off) : bytes(l.ring), kWsAlign);
    return l;
}

Plan plan(const Product &p)
{
    if (!ring_sizes(p) || few_rows(p))
        return plan(p, nullptr);
    const RingWays w = ring_ways(p);
    return plan(p, &w);
}

hipError_t join(const Product &p, hipStream_t s) { return p.splits > 1 ? dgor::launch_join(p, s) : hipSuccess; }

Product as_planned(Product p, const Way &w, void *ws)
{
    p.splits = w.splits;
    p.chunk = w.chunk;
    p.part = (float *)ws;
    return p;
}

// Runs a product; ws has its plan's part bytes.
hipError_t run_product(const Product &q, const Plan &l, void *ws, hipStream_t s)
{
    if (q.M == 0 || q.N == 0)
        return hipSuccess;
    const Way &w = ring_addresses(q) ? l.ring : l.off;
    const Product p = as_planned(q, w, ws);
    const hipError_t err = w.kernel == Kernel::Rows   ? dgor::launch_linear_skinny(p, s)
                           : w.kernel == Kernel::Ring ? dgor::launch_linear_ring(p, w.tile, s)
                                                      : dgor::launch_tile(p, s);
    return err == hipSuccess ? join(p, s) : err;
}

// Both products of a backward pass: each by its own plan, or, where that is
// estimated shorter, in one launch on one tile, so that their workgroups run
// side by side, in one round or in rounds that only the last leaves unfilled.
// In one launch and in two: 1144 rows gated 256 to 3816 (f16) 47.2 and 70.3, 104
// rows gated 88 to 2072 10.1 and 15.3; of at most 64 rows, where the input's
// gradient alone is the few-row kernel's, 24 rows of 224 to 1192 9.6 and 14.3.
// Of 72 drawn passes none takes longer, and the median gains 1.21 times.
struct PairPlan {
    Plan x, w;
    bool together;
    Way way_x, way_w;
    size_t part_x, part;   // x's partial sums together, and room for either way's
};
constexpr double kLaunch = 3.0;   // a launch: its gap on the GPU, or the host's time for it

PairPlan plan_pair(const Product &x, const Product &w, bool want_x, bool want_w)
{
    PairPlan l{};
    if (!want_x || !want_w) {
        if (want_x)
            l.x = plan(x);
        if (want_w)
            l.w = plan(w);
        l.part = want_x ? l.x.part : (want_w ? l.w.part : 0);
        return l;
    }
    const bool rings_x = ring_sizes(x), rings_w = ring_sizes(w);
    const RingWays wx = rings_x ? ring_ways(x) : RingWays{}, ww = rings_w ? ring_ways(w) : RingWays{};
    l.x = plan(x, rings_x ? &wx : nullptr);
    l.w = plan(w, rings_w ? &ww : nullptr);
    l.part = l.x.part > l.w.part ? l.x.part : l.w.part;
    if (!rings_x || !rings_w || l.x.ring.kernel == Kernel::Tile || l.w.ring.kernel != Kernel::Ring ||
        x.M == 0 || x.N == 0 || w.M == 0 || w.N == 0)
        return l;
    double best = l.x.ring.us + l.w.ring.us + kLaunch;
    for (int i = 0; i < kRingTiles; ++i) {
        const RingCost &c = kRings[i];
        if (ring_tile_m(c.tile) == 256)
            continue;
        const Way &a = wx.on[i], &b = ww.on[i];
        const RingTimes ta = times(x, c, a.splits), tb = times(w, c, b.splits);
        const double na = (double)tiles(x, ring_tile_m(c.tile), ring_tile_n(c.tile)) * a.splits;
        const double nb = (double)tiles(w, ring_tile_m(c.tile), ring_tile_n(c.tile)) * b.splits;
        if (na + nb > (1 << 20))
            continue;   // a launch holds 2^32 threads
        double t;
        if (na + nb <= 256) {
            t = ta.alone > tb.alone ? ta.alone : tb.alone;
        } else {
            const double longer = ta.full > tb.full ? ta.full : tb.full;
            t = na + nb <= 256.0 * c.share ? longer
                                           : (na * ta.full + nb * tb.full) / (256.0 * c.share) + 0.5 * longer;
        }
        t += ta.join + tb.join;
        if (t < best)
            best = t, l.together = true, l.way_x = a, l.way_w = b;
    }
    if (l.together) {
        const auto bytes = [](const Product &p, const Way &v) {
            return v.splits <= 1 ? 0 : round_up((size_t)p.nbatch * v.splits * dgor::part_size(p) * sizeof(float), kWsAlign);
        };
        l.part_x = bytes(x, l.way_x);
        const size_t both = l.part_x + bytes(w, l.way_w);
        l.part = both > l.part ? both : l.part;
    }
    return l;
}

hipError_t run_pair(const Product *x, const Product *w, const PairPlan &l, uint8_t *ws, hipStream_t s)
{
    if (x && w && l.together && ring_addresses(*x) && ring_addresses(*w)) {
        const Product a = as_planned(*x, l.way_x, ws), b = as_planned(*w, l.way_w, ws + l.part_x);
        hipError_t err = dgor::launch_linear_ring_pair(b, a, l.way_x.tile, s);
        if (err == hipSuccess)
            err = join(a, s);
        return err == hipSuccess ? join(b, s) : err;
    }
    hipError_t err = hipSuccess;
    if (x)
        err = run_product(*x, l.x, ws, s);
    return w && err == hipSuccess ? run_product(*w, l.w, ws, s) : err;
}

// Whether rows are whole units at strides on them.
bool whole_units(int cols, int ld) { return ld % 8 == 0 && cols % 8 == 0 && ld < (1 << 22); }

// An operand in the workspace or the caller's memory: itself, or its higher
// term and the lower.
struct Held {
    const uint16_t *p, *lo;
};

// Operands that are copied at the front of the workspace, their rows padded
// to whole units for the rings: those whose rows or strides are not.  (1000 x
// 777 by 777 x 1033 on the plain tile, whose loads then fall off dwords: 22
// us; copied, 5 us, and on the ring 16 together.)  With `open` all, as two
// bfloat16 terms of a binary16 operand.
struct Copies {
    dgor::Repack r{};
    size_t at[3] = {}, bytes = 0;
    bool open = false;

    // A stored matrix; returns its index here, -1 where it is used as it is.
    // ld becomes the stride of what the products will read.
    int add(int rows, int cols, int &ld)
    {
        if ((whole_units(cols, ld) && !open) || rows == 0 || cols == 0)
            return -1;
        const int i = r.jobs++;
        r.job[i] = {nullptr, nullptr, nullptr, rows, cols, ld, (int)round_up((size_t)cols, 8), 0};
        at[i] = bytes;
        bytes += (open ? 2 : 1) * size(i);
        ld = r.job[i].ld_to;
        return i;
    }
    // Marks copy i (or none); returns where the operand will be.
    Held use(int i, const uint16_t *from, uint8_t *ws)
    {
        if (i < 0)
            return {from, nullptr};
        dgor::Repack::Job &j = r.job[i];
        j.from = from;
        j.to = (uint16_t *)(ws + at[i]);
        j.lo = open ? (uint16_t *)(ws + at[i] + size(i)) : nullptr;
        return {j.to, j.lo};
    }
    size_t size(int i) const { return round_up((size_t)r.job[i].rows * r.job[i].ld_to * 2, kWsAlign); }
    dgor::Repack marked() const
    {
        dgor::Repack q{};
        for (int i = 0; i < r.jobs; ++i)
            if (r.job[i].from)
                q.job[q.jobs++] = r.job[i];
        return q;
    }
};

Product plain_product(int M, int N, int K)
{
    Product p{};
    p.M = M, p.N = N, p.K = K;
    p.nseg = p.nbatch = p.terms = 1;
    return p;
}

// The three products of a layer with n weights W (1, or 2 for the gated one)
// of K inputs x N outputs; dZ in `terms` (Product).
Product forward_product(int M, int N, int K, int op_w, int ldx, int ldw, bool gated)
{
    Product p = plain_product(M, N, K);
    p.lda = ldx, p.ldb = ldw;
    p.trans_b = op_w == GEMM_OP_T;
    p.gated = gated;
    return p;
}
Product input_gradient_product(int M, int N, int K, int op_w, int lddz, int ldw, int n, int terms)   // dX = sum of dZ W^T
{
    Product p = plain_product(M, K, N);
    p.lda = lddz, p.ldb = ldw;
    p.trans_b = op_w == GEMM_OP_N;
    p.nseg = n * terms;
    p.terms = terms;
    return p;
}
Product weight_gradient_product(int M, int N, int K, int op_w, int ldx, int lddz, int n, int terms)   // X^T dZ, or dZ^T X
{
    Product p = op_w == GEMM_OP_N ? plain_product(K, N, M) : plain_product(N, K, M);
    p.lda = op_w == GEMM_OP_N ? ldx : lddz, p.ldb = op_w == GEMM_OP_N ? lddz : ldx;
    p.trans_a = true;
    p.nbatch = n;
    p.nseg = p.terms = terms;
    return p;
}

// One matrix, or two held alike; `low`: which of the pairs takes the lower term.
dgor::Side side(const Held &a, const Held &b, int low)
{
    const auto bytes = [](const uint16_t *from, const uint16_t *to) { return (long long)((uintptr_t)to - (uintptr_t)from); };
    return {a.p, bytes(a.p, b.p), a.lo ? bytes(a.p, a.lo) : 0, low};
}
// The pairs of a backward product: dZ's (A, or B where `swapped`) with the other
// operand's.
void set_pairs(Product &p, const dgor::Side &dz, const dgor::Side &other, bool swapped)
{
    p.A = swapped ? other : dz;
    p.B = swapped ? dz : other;
}
constexpr int kGradientLow = 1, kOtherLow = 2;   // in Product's order of the terms

// The terms that the gradient of a pre-activation is held in: one where the
// caller asks for its rounding or it needs none, else two, and the products of
// binary16 operands, opened into two themselves, have three.
int gradient_terms(bool bf16, bool exact, int activation)
{
    return exact || (activation & GEMM_ROUND_GRADIENT) ? 1 : bf16 ? 2 : 3;
}

// Whether operands off the units are worth a launch that copies them: not for
// a sum of up to two stages of the plain tile over at most a round of its
// tiles (100 x 100 by 100 x 100: 6.3 us, against 2.9 and 4.6 in two launches,
// which are 7.5 us and 12.1 as a host issues them one after another).
bool worth_copies(const Product &p)
{
    return dgor::product_stages(p) > 2 || tiles(p, dgor::kTile, dgor::kTile) > 512;
}

// The copies of a forward product's A and its one or two B.
void copy_operands(Product &p, Copies &c, int (&copy)[3])
{
    copy[0] = copy[1] = copy[2] = -1;
    if (p.M == 0 || p.N == 0 || few_rows(p))
        return;
    if (!worth_copies(p)) {
        p.units = whole_units(p.K, p.lda) && whole_units(p.trans_b ? p.K : p.N, p.ldb);
        return;
    }
    const int rows = p.trans_b ? p.N : p.K, cols = p.trans_b ? p.K : p.N, ld = p.ldb;
    copy[0] = c.add(p.M, p.K, p.lda);
    copy[1] = c.add(rows, cols, p.ldb);
    if (p.gated) {
        int again = ld;
        copy[2] = c.add(rows, cols, again);
    }
    p.units = true;
}

bool workspace_ok(const void *ws, size_t have, size_t need)
{
    return need == 0 || (ws && have >= need && ((uintptr_t)ws & (kWsAlign - 1)) == 0);
}

int done(hipError_t e) { return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH; }

// ------------------------------------------------------------ dense layer --

int check_linear(const gemm_linear_params *q, Product &p, Plan &l, Copies &c, int (&copy)[3])
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    if (q->M < 0 || q->N < 0 || q->K < 0 || too_large(q->M, q->N) || too_large(q->M, q->K) || too_large(q->K, q->N))
        return GEMM_ERR_INVALID_DIM;
    if (!op_ok(q->op_w) || !ld_ok(q->ldx, q->K) || !ld_ok(q->ldw, q->op_w ? q->K : q->N) || !ld_ok(q->ldy, q->N))
        return GEMM_ERR_INVALID_LAYOUT;
    if (!act_ok(q->activation))
        return GEMM_ERR_INVALID_ACTIVATION;
    p = forward_product(q->M, q->N, q->K, q->op_w, q->ldx, q->ldw, false);
    p.e.act = q->activation;
    copy_operands(p, c, copy);
    l = plan(p);
    return GEMM_OK;
}

int run_linear(bool bf16, const gemm_linear_params *q, const uint16_t *X, const uint16_t *W, const uint16_t *bias,
               const void *R, void *Y, uint16_t *pre, void *ws, size_t ws_bytes, void *stream)
{
    Product p;
    Plan l;
    Copies c;
    int copy[3];
    const int rc = check_linear(q, p, l, c, copy);
    if (rc != GEMM_OK)
        return rc;
    if ((R && !ld_ok(q->ldr, q->N)) || (pre && !ld_ok(q->ldp, q->N)))
        return GEMM_ERR_INVALID_LAYOUT;
    if (missing(X, q->M, q->K) || missing(W, q->K, q->N) || missing(Y, q->M, q->N))
        return GEMM_ERR_NULL_PTR;
    if (q->M == 0 || q->N == 0)
        return GEMM_OK;
    if (!workspace_ok(ws, ws_bytes, c.bytes + l.part))
        return GEMM_ERR_WORKSPACE;
    const int dev = dgor::device_status();
    if (dev != GEMM_OK)
        return dev;
    uint8_t *base = (uint8_t *)ws;
    hipStream_t s = (hipStream_t)stream;
    p.bf16 = bf16;
    const Held Xs = c.use(copy[0], X, base), Ws = c.use(copy[1], W, base);
    p.A = side(Xs, Xs, 0);
    p.B = side(Ws, Ws, 0);
    p.e.Y = Y, p.e.ldy = q->ldy, p.e.y_f32 = q->y_f32 != 0;
    p.e.bias = bias;
    p.e.R = R, p.e.ldr = q->ldr;
    p.e.pre = pre, p.e.ldp = q->ldp;
    const hipError_t err = dgor::launch_repack(c.marked(), s);
    return done(err == hipSuccess ? run_product(p, l, base + c.bytes, s) : err);
}

// Workspace of the dense layer's backward pass: copies, dZ or its two terms, the
// column sums of each row block, and the partial sums of whichever product is
// running.
struct BackwardLayout {
    Copies c;
    PairPlan products;
    int copy_dy, copy_x, copy_w;
    int terms, lddz;
    size_t dz, dz_lo, sums, part, bytes;   // offsets, and the whole size
};

int row_blocks(int M, int N) { return ceil_div(M, dgor::grad_rows(M, N)); }

void lay_out(const gemm_linear_backward_params *q, bool bf16, Product &px, Product &pw, BackwardLayout &l)
{
    // slopes of 0 and 1 leave dY's values as they are
    const int kind = act_of(q->activation);
    const bool act = kind != GEMM_ACT_NONE, t = q->op_w == GEMM_OP_T;
    const bool want_x = wants_input(q->activation), want_w = wants_weight(q->activation);
    l = BackwardLayout{};
    l.terms = gradient_terms(bf16, kind <= GEMM_ACT_RELU, q->activation);
    l.c.open = l.terms == 3;
    int ldx = q->ldx, ldw = q->ldw;
    l.lddz = act ? (int)round_up((size_t)q->N, 8) : q->lddy;
    px = input_gradient_product(q->M, q->N, q->K, q->op_w, l.lddz, ldw, 1, l.terms);
    pw = weight_gradient_product(q->M, q->N, q->K, q->op_w, ldx, l.lddz, 1, l.terms);
    const bool for_x = want_x && !few_rows(px) && (l.c.open || worth_copies(px));
    const bool for_w = want_w && (l.c.open || worth_copies(pw));
    l.copy_dy = !act && (for_x || for_w) ? l.c.add(q->M, q->N, l.lddz) : -1;
    l.copy_x = for_w ? l.c.add(q->M, q->K, ldx) : -1;
    l.copy_w = for_x ? l.c.add(t ? q->N : q->K, t ? q->K : q->N, ldw) : -1;
    px = input_gradient_product(q->M, q->N, q->K, q->op_w, l.lddz, ldw, 1, l.terms);
    pw = weight_gradient_product(q->M, q->N, q->K, q->op_w, ldx, l.lddz, 1, l.terms);
    const bool dz_units = act || for_x || for_w || whole_units(q->N, l.lddz);
    px.opened = l.c.open && for_x;
    pw.opened = l.c.open;
    px.units = dz_units && (for_x || (!l.c.open && whole_units(t ? q->K : q->N, ldw)));
    pw.units = dz_units && (for_w || whole_units(q->K, ldx));
    const size_t dz_bytes = act && (want_x || want_w) ? round_up((size_t)q->M * l.lddz * 2, kWsAlign) : 0;
    l.dz = l.c.bytes;
    l.dz_lo = l.dz + dz_bytes;
    l.sums = l.dz_lo + (l.terms > 1 ? dz_bytes : 0);
    l.part = l.sums + round_up((size_t)row_blocks(q->M, q->N) * q->N * sizeof(float), kWsAlign);
    l.products = plan_pair(px, pw, want_x, want_w);
    l.bytes = l.part + l.products.part;
}

// Checks, products and layout of one format, and the workspace's size for
// either, or for the one that the flags name.
int check_linear_backward(const gemm_linear_backward_params *q, bool bf16, Product &px, Product &pw, BackwardLayout &l,
                          size_t &bytes)
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    if (q->M < 0 || q->N < 0 || q->K < 0 || too_large(q->M, q->N) || too_large(q->M, q->K) || too_large(q->K, q->N))
        return GEMM_ERR_INVALID_DIM;
    if (!op_ok(q->op_w) || !ld_ok(q->lddy, q->N))
        return GEMM_ERR_INVALID_LAYOUT;
    if (!act_ok(act_of(q->activation)))
        return GEMM_ERR_INVALID_ACTIVATION;
    bytes = 0;
    // where the formats differ
    if (takes(!bf16, q->activation) && gradient_terms(false, act_of(q->activation) <= GEMM_ACT_RELU, q->activation) > 1) {
        lay_out(q, !bf16, px, pw, l);
        bytes = l.bytes;
    }
    lay_out(q, bf16, px, pw, l);
    bytes = l.bytes > bytes ? l.bytes : bytes;
    return GEMM_OK;
}

int run_linear_backward(bool bf16, const gemm_linear_backward_params *q, const uint16_t *dY, const uint16_t *X,
                        const uint16_t *W, const uint16_t *pre, uint16_t *dX, uint16_t *dW, uint16_t *dbias, void *ws,
                        size_t ws_bytes, void *stream)
{
    Product px, pw;
    BackwardLayout l;
    size_t need;
    const int rc = check_linear_backward(q, bf16, px, pw, l, need);
    if (rc != GEMM_OK)
        return rc;
    if (!takes(bf16, q->activation) || (dX && !wants_input(q->activation)) || (dW && !wants_weight(q->activation)))
        return GEMM_ERR_INVALID_ACTIVATION;
    const int kind = act_of(q->activation);
    const bool act = kind != GEMM_ACT_NONE;
    const int w_row = q->op_w ? q->K : q->N;
    if ((dX && (!ld_ok(q->ldw, w_row) || !ld_ok(q->lddx, q->K))) ||
        (dW && (!ld_ok(q->ldx, q->K) || !ld_ok(q->lddw, w_row))) || (act && !ld_ok(q->ldp, q->N)))
        return GEMM_ERR_INVALID_LAYOUT;
    if (missing(dY, q->M, q->N) || (act && missing(pre, q->M, q->N)) || (dX && missing(W, q->K, q->N)) ||
        (dW && missing(X, q->M, q->K)))
        return GEMM_ERR_NULL_PTR;
    if (!workspace_ok(ws, ws_bytes, need))
        return GEMM_ERR_WORKSPACE;
    const int dev = dgor::device_status();
    if (dev != GEMM_OK)
        return dev;
    hipStream_t s = (hipStream_t)stream;
    uint8_t *base = (uint8_t *)ws;
    const int blocks = row_blocks(q->M, q->N);
    float *sums = dbias && blocks != 1 ? (float *)(base + l.sums) : nullptr;
    px.bf16 = pw.bf16 = bf16 || l.terms > 1;
    px.e.y_f16 = pw.e.y_f16 = !bf16 && l.terms > 1;
    Held dZ = l.c.use(dX || dW ? l.copy_dy : -1, dY, base);
    const Held Xs = l.c.use(dW ? l.copy_x : -1, X, base), Ws = l.c.use(dX ? l.copy_w : -1, W, base);
    hipError_t err;
    if (q->M > 0 && q->N > 0 && ((act && (dX || dW)) || dbias)) {
        uint16_t *out = act && (dX || dW) ? (uint16_t *)(base + l.dz) : nullptr;
        uint16_t *lo = out && l.terms > 1 ? (uint16_t *)(base + l.dz_lo) : nullptr;
        err = dgor::launch_act_grad(q->M, q->N, dY, q->lddy, act ? pre : nullptr, q->ldp, out, lo, l.lddz, kind, sums,
                                    blocks == 1 ? dbias : nullptr, l.c.marked(), bf16, s);
        if (out)
            dZ = {out, lo};
    } else {
        err = dgor::launch_repack(l.c.marked(), s);
    }
    // no rows: an empty sum, no workspace
    if (err == hipSuccess && dbias && blocks != 1 && q->N > 0)
        err = dgor::launch_sum_blocks(blocks, q->N, sums, dbias, bf16, s);
    if (err != hipSuccess)
        return GEMM_ERR_LAUNCH;
    if (dX) {
        set_pairs(px, side(dZ, dZ, kGradientLow), side(Ws, Ws, kOtherLow), false);
        px.e.Y = dX, px.e.ldy = q->lddx;
    }
    if (dW) {
        set_pairs(pw, side(dZ, dZ, kGradientLow), side(Xs, Xs, kOtherLow), q->op_w == GEMM_OP_N);
        pw.e.Y = dW, pw.e.ldy = q->lddw;
    }
    return done(run_pair(dX ? &px : nullptr, dW ? &pw : nullptr, l.products, base + l.part, s));
}

// ---------------------------------------------------- gated up-projection --

int check_gated(const gemm_gated_params *q, Product &p, Plan &l, Copies &c, int (&copy)[3])
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    if (q->M < 0 || q->F < 0 || q->K < 0 || too_large(q->M, q->F) || too_large(q->M, q->K) || too_large(q->K, q->F))
        return GEMM_ERR_INVALID_DIM;
    if (!op_ok(q->op_w) || !ld_ok(q->ldx, q->K) || !ld_ok(q->ldw, q->op_w ? q->K : q->F) || !ld_ok(q->ldh, q->F))
        return GEMM_ERR_INVALID_LAYOUT;
    if (!act_ok(q->activation))
        return GEMM_ERR_INVALID_ACTIVATION;
    p = forward_product(q->M, q->F, q->K, q->op_w, q->ldx, q->ldw, true);
    p.e.act = q->activation;
    copy_operands(p, c, copy);
    l = plan(p);
    return GEMM_OK;
}

int run_gated(bool bf16, const gemm_gated_params *q, const uint16_t *X, const uint16_t *Wg, const uint16_t *Wu,
              uint16_t *H, uint16_t *G, uint16_t *U, void *ws, size_t ws_bytes, void *stream)
{
    Product p;
    Plan l;
    Copies c;
    int copy[3];
    const int rc = check_gated(q, p, l, c, copy);
    if (rc != GEMM_OK)
        return rc;
    if (G && !ld_ok(q->ldp, q->F))
        return GEMM_ERR_INVALID_LAYOUT;
    if (missing(X, q->M, q->K) || missing(Wg, q->K, q->F) || missing(Wu, q->K, q->F) || missing(H, q->M, q->F) ||
        (G != nullptr) != (U != nullptr))
        return GEMM_ERR_NULL_PTR;
    if (q->M == 0 || q->F == 0)
        return GEMM_OK;
    if (!workspace_ok(ws, ws_bytes, c.bytes + l.part))
        return GEMM_ERR_WORKSPACE;
    const int dev = dgor::device_status();
    if (dev != GEMM_OK)
        return dev;
    uint8_t *base = (uint8_t *)ws;
    hipStream_t s = (hipStream_t)stream;
    p.bf16 = bf16;
    const Held Xs = c.use(copy[0], X, base), Gs = c.use(copy[1], Wg, base), Us = c.use(copy[2], Wu, base);
    p.A = side(Xs, Xs, 0);
    p.B = side(Gs, Us, 0);
    p.e.Y = H, p.e.ldy = q->ldh;
    p.e.pre = G, p.e.pre2 = U, p.e.ldp = q->ldp;
    const hipError_t err = dgor::launch_repack(c.marked(), s);
    return done(err == hipSuccess ? run_product(p, l, base + c.bytes, s) : err);
}

// Workspace of the gated backward pass: copies, dG and dU or their terms, then
// the partial sums of whichever product is running.
struct GatedBackwardLayout {
    Copies c;
    PairPlan products;
    int copy_x, copy_wg, copy_wu;
    int terms, ldd;
    size_t d, d_bytes, part, bytes;   // dG, dU and their lower terms, each d_bytes after the one before
};

void lay_out(const gemm_gated_backward_params *q, bool bf16, Product &px, Product &pw, GatedBackwardLayout &l)
{
    l = GatedBackwardLayout{};
    l.terms = gradient_terms(bf16, false, q->activation);
    l.c.open = l.terms == 3;
    l.ldd = (int)round_up((size_t)q->F, 8);
    const bool t = q->op_w == GEMM_OP_T;
    const bool want_x = wants_input(q->activation), want_w = wants_weight(q->activation);
    int ldx = q->ldx, ldw = q->ldw, ldu = q->ldw;
    px = input_gradient_product(q->M, q->F, q->K, q->op_w, l.ldd, ldw, 2, l.terms);
    pw = weight_gradient_product(q->M, q->F, q->K, q->op_w, ldx, l.ldd, 2, l.terms);
    const bool for_x = want_x && !few_rows(px) && (l.c.open || worth_copies(px));
    const bool for_w = want_w && (l.c.open || worth_copies(pw));
    l.copy_x = for_w ? l.c.add(q->M, q->K, ldx) : -1;
    l.copy_wg = for_x ? l.c.add(t ? q->F : q->K, t ? q->K : q->F, ldw) : -1;
    l.copy_wu = for_x ? l.c.add(t ? q->F : q->K, t ? q->K : q->F, ldu) : -1;
    px.ldb = ldw;
    pw = weight_gradient_product(q->M, q->F, q->K, q->op_w, ldx, l.ldd, 2, l.terms);
    px.opened = l.c.open && for_x;
    pw.opened = l.c.open;
    px.units = for_x || (!l.c.open && whole_units(t ? q->K : q->F, ldw));
    pw.units = for_w || whole_units(q->K, ldx);
    l.d = l.c.bytes;
    l.d_bytes = round_up((size_t)q->M * l.ldd * 2, kWsAlign);
    l.part = l.d + (l.terms > 1 ? 4 : 2) * l.d_bytes;
    l.products = plan_pair(px, pw, want_x, want_w);
    l.bytes = want_x || want_w ? l.part + l.products.part : 0;
}

int check_gated_backward(const gemm_gated_backward_params *q, bool bf16, Product &px, Product &pw,
                         GatedBackwardLayout &l, size_t &bytes)
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    if (q->M < 0 || q->F < 0 || q->K < 0 || too_large(q->M, q->F) || too_large(q->M, q->K) || too_large(q->K, q->F))
        return GEMM_ERR_INVALID_DIM;
    if (!op_ok(q->op_w) || !ld_ok(q->lddh, q->F) || !ld_ok(q->ldp, q->F))
        return GEMM_ERR_INVALID_LAYOUT;
    if (!act_ok(act_of(q->activation)))
        return GEMM_ERR_INVALID_ACTIVATION;
    bytes = 0;
    if (takes(!bf16, q->activation) && gradient_terms(false, false, q->activation) > 1) {   // the formats differ
        lay_out(q, !bf16, px, pw, l);
        bytes = l.bytes;
    }
    lay_out(q, bf16, px, pw, l);
    bytes = l.bytes > bytes ? l.bytes : bytes;
    return GEMM_OK;
}

int run_gated_backward(bool bf16, const gemm_gated_backward_params *q, const uint16_t *dH, const uint16_t *X,
                       const uint16_t *Wg, const uint16_t *Wu, const uint16_t *G, const uint16_t *U, uint16_t *dX,
                       uint16_t *dWg, uint16_t *dWu, void *ws, size_t ws_bytes, void *stream)
{
    Product px, pw;
    GatedBackwardLayout l;
    size_t need;
    const int rc = check_gated_backward(q, bf16, px, pw, l, need);
    if (rc != GEMM_OK)
        return rc;
    if (!takes(bf16, q->activation) || (dX && !wants_input(q->activation)) || (dWg && !wants_weight(q->activation)))
        return GEMM_ERR_INVALID_ACTIVATION;
    const int w_row = q->op_w ? q->K : q->F;
    if ((dX && (!ld_ok(q->ldw, w_row) || !ld_ok(q->lddx, q->K))) ||
        (dWg && (!ld_ok(q->ldx, q->K) || !ld_ok(q->lddw, w_row))))
        return GEMM_ERR_INVALID_LAYOUT;
    if (missing(dH, q->M, q->F) || missing(G, q->M, q->F) || missing(U, q->M, q->F) ||
        (dX && (missing(Wg, q->K, q->F) || missing(Wu, q->K, q->F))) || (dWg && missing(X, q->M, q->K)) ||
        (dWg != nullptr) != (dWu != nullptr))
        return GEMM_ERR_NULL_PTR;
    if (!dX && !dWg)
        return GEMM_OK;
    if (!workspace_ok(ws, ws_bytes, need))
        return GEMM_ERR_WORKSPACE;
    const int dev = dgor::device_status();
    if (dev != GEMM_OK)
        return dev;
    hipStream_t s = (hipStream_t)stream;
    uint8_t *base = (uint8_t *)ws;
    const auto part = [&](int i) { return (uint16_t *)(base + l.d + i * l.d_bytes); };
    const bool two = l.terms > 1;
    const dgor::GateGrads d{{part(0), two ? part(2) : nullptr}, {part(1), two ? part(3) : nullptr}};
    px.bf16 = pw.bf16 = bf16 || two;
    px.e.y_f16 = pw.e.y_f16 = !bf16 && two;
    const Held Xs = l.c.use(dWg ? l.copy_x : -1, X, base);
    const Held Gs = l.c.use(dX ? l.copy_wg : -1, Wg, base), Us = l.c.use(dX ? l.copy_wu : -1, Wu, base);
    const hipError_t err = q->M > 0 && q->F > 0
                               ? dgor::launch_gate_grad(q->M, q->F, dH, q->lddh, G, U, q->ldp, d, l.ldd,
                                                        act_of(q->activation), l.c.marked(), bf16, s)
                               : dgor::launch_repack(l.c.marked(), s);
    if (err != hipSuccess)
        return GEMM_ERR_LAUNCH;
    const dgor::Side dz = side({d.g[0], d.g[1]}, {d.u[0], d.u[1]}, kGradientLow);
    if (dX) {
        set_pairs(px, dz, side(Gs, Us, kOtherLow), false);
        px.e.Y = dX, px.e.ldy = q->lddx;
    }
    if (dWg) {
        set_pairs(pw, dz, side(Xs, Xs, kOtherLow), q->op_w == GEMM_OP_N);
        pw.e.Y = dWg, pw.Y1 = dWu, pw.e.ldy = q->lddw;
    }
    return done(run_pair(dX ? &px : nullptr, dWg ? &pw : nullptr, l.products, base + l.part, s));
}

}  // namespace

extern "C" {

int gemm_linear_workspace(const gemm_linear_params *params, size_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_NULL_PTR;
    Product p;
    Plan l;
    Copies c;
    int copy[3];
    const int rc = check_linear(params, p, l, c, copy);
    if (rc == GEMM_OK)
        *bytes = p.M && p.N ? c.bytes + l.part : 0;
    return rc;
}
int gemm_linear_f16(const gemm_linear_params *params, const uint16_t *X, const uint16_t *W, const uint16_t *bias,
                    const void *R, void *Y, uint16_t *pre, void *workspace, size_t workspace_bytes, void *stream)
{
    return run_linear(false, params, X, W, bias, R, Y, pre, workspace, workspace_bytes, stream);
}
int gemm_linear_bf16(const gemm_linear_params *params, const uint16_t *X, const uint16_t *W, const uint16_t *bias,
                     const void *R, void *Y, uint16_t *pre, void *workspace, size_t workspace_bytes, void *stream)
{
    return run_linear(true, params, X, W, bias, R, Y, pre, workspace, workspace_bytes, stream);
}

int gemm_linear_backward_workspace(const gemm_linear_backward_params *params, size_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_NULL_PTR;
    Product px, pw;
    BackwardLayout l;
    size_t need;
    const int rc = check_linear_backward(params, !params || takes(true, params->activation), px, pw, l, need);
    if (rc == GEMM_OK)
        *bytes = need;
    return rc;
}
int gemm_linear_backward_f16(const gemm_linear_backward_params *params, const uint16_t *dY, const uint16_t *X,
                             const uint16_t *W, const uint16_t *pre, uint16_t *dX, uint16_t *dW, uint16_t *dbias,
                             void *workspace, size_t workspace_bytes, void *stream)
{
    return run_linear_backward(false, params, dY, X, W, pre, dX, dW, dbias, workspace, workspace_bytes, stream);
}
int gemm_linear_backward_bf16(const gemm_linear_backward_params *params, const uint16_t *dY, const uint16_t *X,
                              const uint16_t *W, const uint16_t *pre, uint16_t *dX, uint16_t *dW, uint16_t *dbias,
                              void *workspace, size_t workspace_bytes, void *stream)
{
    return run_linear_backward(true, params, dY, X, W, pre, dX, dW, dbias, workspace, workspace_bytes, stream);
}

int gemm_gated_workspace(const gemm_gated_params *params, size_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_NULL_PTR;
    Product p;
    Plan l;
    Copies c;
    int copy[3];
    const int rc = check_gated(params, p, l, c, copy);
    if (rc == GEMM_OK)
        *bytes = p.M && p.N ? c.bytes + l.part : 0;
    return rc;
}
int gemm_gated_f16(const gemm_gated_params *params, const uint16_t *X, const uint16_t *Wg, const uint16_t *Wu,
                   uint16_t *H, uint16_t *G, uint16_t *U, void *workspace, size_t workspace_bytes, void *stream)
{
    return run_gated(false, params, X, Wg, Wu, H, G, U, workspace, workspace_bytes, stream);
}
int gemm_gated_bf16(const gemm_gated_params *params, const uint16_t *X, const uint16_t *Wg, const uint16_t *Wu,
                    uint16_t *H, uint16_t *G, uint16_t *U, void *workspace, size_t workspace_bytes, void *stream)
{
    return run_gated(true, params, X, Wg, Wu, H, G, U, workspace, workspace_bytes, stream);
}

int gemm_gated_backward_workspace(const gemm_gated_backward_params *params, size_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_NULL_PTR;
    Product px, pw;
    GatedBackwardLayout l;
    size_t need;
    const int rc = check_gated_backward(params, !params || takes(true, params->activation), px, pw, l, need);
    if (rc == GEMM_OK)
        *bytes = need;
    return rc;
}
int gemm_gated_backward_f16(const gemm_gated_backward_params *params, const uint16_t *dH, const uint16_t *X,
                            const uint16_t *Wg, const uint16_t *Wu, const uint16_t *G, const uint16_t *U,
                            uint16_t *dX, uint16_t *dWg, uint16_t *dWu, void *workspace, size_t workspace_bytes,
                            void *stream)
{
    return run_gated_backward(false, params, dH, X, Wg, Wu, G, U, dX, dWg, dWu, workspace, workspace_bytes, stream);
}
int gemm_gated_backward_bf16(const gemm_gated_backward_params *params, const uint16_t *dH, const uint16_t *X,
                             const uint16_t *Wg, const uint16_t *Wu, const uint16_t *G, const uint16_t *U,
                             uint16_t *dX, uint16_t *dWg, uint16_t *dWu, void *workspace, size_t workspace_bytes,
                             void *stream)
{
    return run_gated_backward(true, params, dH, X, Wg, Wu, G, U, dX, dWg, dWu, workspace, workspace_bytes, stream);
}

}  // extern "C"
