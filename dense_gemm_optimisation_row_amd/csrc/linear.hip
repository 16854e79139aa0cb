// C entry points of the dense layer and the gated up-projection (declared in
// include/gemm.h): argument checks, choice of kernel, workspace layout.
// Host code only; the kernels live in linear_skinny.hip, linear_ring.hip,
// linear_tile.hip and act_grad.hip.
#include <stdint.h>

#include "linear.h"

namespace {

using dgor::Epilogue;
using dgor::Product;

constexpr size_t kWsAlign = 256;
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// A launch holds 2^32 threads: at most 2^22 tiles of 128 x 64, twice.
bool too_large(long long rows, long long cols) { return (rows + 127) / 128 * ((cols + 63) / 64) > (1LL << 22); }
bool ld_ok(int ld, int row) { return ld >= (row > 1 ? row : 1); }
bool op_ok(int op) { return op == GEMM_OP_N || op == GEMM_OP_T; }
bool act_ok(int act) { return act >= GEMM_ACT_NONE && act <= GEMM_ACT_SILU; }
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

long long tiles(const Product &p, int tm, int tn)
{
    return (long long)ceil_div(p.M, tm) * ceil_div(p.N, p.gated ? tn / 2 : tn) * p.nbatch;
}

// Whether the few-row kernel takes a product.
bool few_rows(const Product &p)
{
    return !p.trans_a && p.nbatch == 1 && p.M <= dgor::kSkinnyRows && dgor::spans_a_unit(p);
}

// Whether sizes and strides let the rings run (the addresses apart).
bool ring_sizes(const Product &p)
{
    const auto ok = [](int ld) { return ld % 8 == 0 && ld < (1 << 22); };
    return p.units && ok(p.lda) && ok(p.ldb);
}
bool ring_addresses(const Product &p)
{
    return (((uintptr_t)p.A[0] | (uintptr_t)p.A[1] | (uintptr_t)p.B[0] | (uintptr_t)p.B[1]) & 15) == 0;
}

void split(const Product &p, long long parts, Way &w)
{
    w.splits = 1, w.chunk = 0;
    if (parts > 1) {
        w.chunk = ceil_div(dgor::product_stages(p), parts);
        w.splits = ceil_div(dgor::product_stages(p), w.chunk);
    }
}

// Time of a product on a ring's tile with its sum in `parts`.  Up to `share`
// workgroups of the tile run on a compute unit at once.  A round of at most one
// a unit takes ends + alone for each 32 k, a full one ends_full + full each.
// Parts are written in FP32 and joined by another launch.  Microseconds, fitted
// to 16 to 4096 workgroups of each tile and sums of 256 to 4096 (BF16, K x N):
// within 10% of the times measured.  Full rates: 1470, 1280, 1180, 890 and
// 570 TFLOP/s.  An activation of exponentials adds what its outputs take on the
// vector ALUs: 9 us for 256 x 256 (GELU, 4096 x 8192 outputs of 4096: 222 us,
// 204 without).
struct RingCost {
    dgor::RingTile tile;
    int share;
    double ends, alone, ends_full, full;
    double halves;   // times as long a stage whose loads take half lines
};
constexpr RingCost kRings[] = {
    {dgor::kRing256, 1, 14.5, 0.73, 14.5, 0.73, 1.0},
    {dgor::kRing256x128, 1, 9.8, 0.42, 9.8, 0.42, 1.3},
    {dgor::kRing128, 2, 6.8, 0.295, 7.5, 0.455, 1.17},
    {dgor::kRing128x64, 2, 4.8, 0.243, 6.2, 0.33, 1.12},
    {dgor::kRing64, 2, 4.0, 0.158, 4.2, 0.243, 1.08},
};
constexpr int kSplitRows = 40;   // stages of 64 k from which few rows' sums over a K x N matrix are split
constexpr double kJoinLaunch = 4.5, kJoinBytes = 8e6;   // and a microsecond's bytes
// Weights that the few-row kernel reads in a microsecond, past 3 us: 33.5 MB
// 11 us, 134 MB 28 us.
constexpr double kRowsBytes = 5e6;
struct RingTimes {
    double alone, full, join;   // a round of one tile a unit, a full one, joining the parts
};
RingTimes times(const Product &p, const RingCost &c, int parts)
{
    // half lines: B as N x K, and each of two matrices' 32 columns
    const bool halves = p.trans_b || (p.gated && ring_tile_n(c.tile) == 64);
    const double stages = 2.0 * dgor::product_stages(p) / parts * (halves ? c.halves : 1.0);
    // an activation's time for a workgroup's outputs
    const double act = p.e.act > GEMM_ACT_RELU && parts == 1
                           ? 9.0 * ring_tile_m(c.tile) * ring_tile_n(c.tile) / (p.gated ? 131072 : 65536)
                           : 0.0;
    return {c.ends + stages * c.alone + act, c.ends_full + stages * c.full + act * c.share,
            parts > 1 ? kJoinLaunch + 8.0 * parts * (p.gated ? 2 : p.nbatch) * p.M * p.N / kJoinBytes : 0.0};
}
double microseconds(const Product &p, const RingCost &c, int parts)
{
    const long long n = tiles(p, ring_tile_m(c.tile), ring_tile_n(c.tile)) * parts;
    const long long rounds = n / (256LL * c.share), rest = n % (256LL * c.share);
    const RingTimes t = times(p, c, parts);
    return rounds * t.full + (rest == 0 ? 0.0 : rest <= 256 ? t.alone : t.full) + t.join;
}

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
        const double t = microseconds(p, c, parts);
        if (parts == 1 || t < w.us)
            w.us = t, best = parts;
    }
    split(p, best, w);
    return w;
}

Way choose(const Product &p, bool ring)
{
    Way w{Kernel::Rows, dgor::kRing64, 1, 0, 0};
    const int stages = dgor::product_stages(p);
    if (few_rows(p)) {
        // a K x N matrix with a long sum and too few columns for the compute
        // units: parts of at least eight stages, one for each wavefront
        const long long strips = ceil_div(p.N, dgor::skinny_strip(p, true));
        if (!p.trans_b && stages >= kSplitRows && strips < 256) {
            long long want = (256 + strips - 1) / strips;
            want = want < stages / 8 ? want : stages / 8;
            split(p, want < 32 ? want : 32, w);
        }
        w.us = 3.0 + 2.0 * p.nseg * p.K * p.N / kRowsBytes + (w.splits > 1 ? kJoinLaunch : 0.0);
        return w;
    }
    if (ring) {
        for (const RingCost &c : kRings) {
            const Way v = best_on(p, c);
            if (w.kernel != Kernel::Ring || v.us < w.us)
                w = v;
        }
        return w;
    }
    // the plain tile: split until two workgroups a compute unit, keeping at
    // least four stages a part
    w.kernel = Kernel::Tile;
    const long long n = tiles(p, dgor::kTile, dgor::kTile);
    if (n > 0 && n < 256 && stages >= 8) {
        long long want = 512 / n;
        want = want < stages / 4 ? want : stages / 4;
        split(p, want < 16 ? want : 16, w);
    }
    return w;
}

// How a product runs off and on the rings, as the operands' addresses will
// have it, and the bytes of its FP32 partial sums either way.
struct Plan {
    Way off, ring;
    size_t part;
};
Plan plan(const Product &p)
{
    const auto bytes = [&](const Way &w) {
        return w.splits <= 1 ? 0 : (size_t)(p.gated ? 2 : p.nbatch) * w.splits * dgor::part_size(p) * sizeof(float);
    };
    Plan l;
    l.off = choose(p, false);
    l.ring = ring_sizes(p) ? choose(p, true) : l.off;
    l.part = round_up(bytes(l.off) > bytes(l.ring) ? bytes(l.off) : bytes(l.ring), kWsAlign);
    return l;
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
// In one launch and in two: 528 rows of 2752 to 791 outputs 25.6 us and 35.2,
// 3344 rows gated 684 to 640 39.6 and 52.7, 2960 rows gated 244 to 5614 100 and
// 116, 3266 rows of 3512 to 64 30.7 and 38.4; of at most 64 rows, where the
// input's gradient alone is the few-row kernel's, 16 rows of 248 to 640 12.9
// and 15.7.  Of 150 drawn passes none takes longer.
struct PairPlan {
    Plan x, w;
    bool together;
    Way way_x, way_w;
    size_t part_x, part;   // x's partial sums together, and room for either way's
};
constexpr double kLaunch = 3.0;   // a launch: its gap on the GPU, or the host's time for it

PairPlan plan_pair(const Product &x, const Product &w)
{
    PairPlan l{};
    l.x = plan(x);
    l.w = plan(w);
    l.part = l.x.part > l.w.part ? l.x.part : l.w.part;
    if (!ring_sizes(x) || !ring_sizes(w) || l.x.ring.kernel == Kernel::Tile || l.w.ring.kernel != Kernel::Ring ||
        x.M == 0 || x.N == 0 || w.M == 0 || w.N == 0)
        return l;
    double best = l.x.ring.us + l.w.ring.us + kLaunch;
    for (const RingCost &c : kRings) {
        if (ring_tile_m(c.tile) == 256)
            continue;
        const Way a = best_on(x, c), b = best_on(w, c);
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

// Operands that are copied at the front of the workspace, their rows padded
// to whole units for the rings: those whose rows or strides are not.  (1000 x
// 777 by 777 x 1033 on the plain tile, whose loads then fall off dwords: 22
// us; copied, 5 us, and on the ring 16 together.)
struct Copies {
    dgor::Repack r{};
    size_t at[3] = {}, bytes = 0;
    bool units = true;   // the operands' rows are whole units, or padded to them

    // A stored matrix; returns its index here, -1 where it is used as it is.
    // ld becomes the stride of what the products will read.
    int add(int rows, int cols, int &ld)
    {
        if (whole_units(cols, ld) || rows == 0 || cols == 0)
            return -1;
        if ((long long)rows * ceil_div(cols, 8) >= (1LL << 30)) {   // a launch's units are counted in 32 bits
            units = false;
            return -1;
        }
        const int i = r.jobs++;
        r.job[i] = {nullptr, nullptr, rows, cols, ld, (int)round_up((size_t)cols, 8), 0u};
        at[i] = bytes;
        bytes += round_up((size_t)rows * r.job[i].ld_to * 2, kWsAlign);
        ld = r.job[i].ld_to;
        return i;
    }
    // Marks copy i (or none); returns where the operand will be.
    const uint16_t *use(int i, const uint16_t *from, uint8_t *ws)
    {
        if (i < 0)
            return from;
        r.job[i].from = from;
        r.job[i].to = (uint16_t *)(ws + at[i]);
        return r.job[i].to;
    }
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
    p.nseg = p.nbatch = 1;
    return p;
}

// The three products of a layer with n weights W (1, or 2 for the gated one)
// of K inputs x N outputs.
Product forward_product(int M, int N, int K, int op_w, int ldx, int ldw, bool gated)
{
    Product p = plain_product(M, N, K);
    p.lda = ldx, p.ldb = ldw;
    p.trans_b = op_w == GEMM_OP_T;
    p.gated = gated;
    return p;
}
Product input_gradient_product(int M, int N, int K, int op_w, int lddz, int ldw, int n)   // dX = sum of dZ W^T
{
    Product p = plain_product(M, K, N);
    p.lda = lddz, p.ldb = ldw;
    p.trans_b = op_w == GEMM_OP_N;
    p.nseg = n;
    return p;
}
Product weight_gradient_product(int M, int N, int K, int op_w, int ldx, int lddz, int n)   // X^T dZ, or dZ^T X
{
    Product p = op_w == GEMM_OP_N ? plain_product(K, N, M) : plain_product(N, K, M);
    p.lda = op_w == GEMM_OP_N ? ldx : lddz, p.ldb = op_w == GEMM_OP_N ? lddz : ldx;
    p.trans_a = true;
    p.nbatch = n;
    return p;
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
    p.units = c.units;
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
    p.A[0] = p.A[1] = c.use(copy[0], X, base);
    p.B[0] = p.B[1] = c.use(copy[1], W, base);
    p.e.Y = Y, p.e.ldy = q->ldy, p.e.y_f32 = q->y_f32 != 0;
    p.e.bias = bias;
    p.e.R = R, p.e.ldr = q->ldr;
    p.e.pre = pre, p.e.ldp = q->ldp;
    const hipError_t err = dgor::launch_repack(c.marked(), s);
    return done(err == hipSuccess ? run_product(p, l, base + c.bytes, s) : err);
}

// Workspace of the dense layer's backward pass: copies, dZ, the column sums of
// each row block, and the partial sums of whichever product is running.
struct BackwardLayout {
    Copies c;
    PairPlan products;
    int copy_dy, copy_x, copy_w;
    int lddz;
    size_t dz, sums, part, bytes;   // offsets, and the whole size
};

int row_blocks(int M, int N) { return ceil_div(M, dgor::grad_rows(M, N)); }

int check_linear_backward(const gemm_linear_backward_params *q, Product &px, Product &pw, BackwardLayout &l)
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    if (q->M < 0 || q->N < 0 || q->K < 0 || too_large(q->M, q->N) || too_large(q->M, q->K) || too_large(q->K, q->N))
        return GEMM_ERR_INVALID_DIM;
    if (!op_ok(q->op_w) || !ld_ok(q->lddy, q->N))
        return GEMM_ERR_INVALID_LAYOUT;
    if (!act_ok(q->activation))
        return GEMM_ERR_INVALID_ACTIVATION;
    const bool act = q->activation != GEMM_ACT_NONE, t = q->op_w == GEMM_OP_T;
    int ldx = q->ldx, ldw = q->ldw;
    l.lddz = act ? (int)round_up((size_t)q->N, 8) : q->lddy;
    px = input_gradient_product(q->M, q->N, q->K, q->op_w, l.lddz, ldw, 1);
    pw = weight_gradient_product(q->M, q->N, q->K, q->op_w, ldx, l.lddz, 1);
    const bool for_x = !few_rows(px) && worth_copies(px), for_w = worth_copies(pw);
    l.copy_dy = !act && (for_x || for_w) ? l.c.add(q->M, q->N, l.lddz) : -1;
    l.copy_x = for_w ? l.c.add(q->M, q->K, ldx) : -1;
    l.copy_w = for_x ? l.c.add(t ? q->N : q->K, t ? q->K : q->N, ldw) : -1;
    px = input_gradient_product(q->M, q->N, q->K, q->op_w, l.lddz, ldw, 1);
    pw = weight_gradient_product(q->M, q->N, q->K, q->op_w, ldx, l.lddz, 1);
    const bool dz_units = act || for_x || for_w || whole_units(q->N, l.lddz);
    px.units = l.c.units && dz_units && (for_x || whole_units(t ? q->K : q->N, ldw));
    pw.units = l.c.units && dz_units && (for_w || whole_units(q->K, ldx));
    l.dz = l.c.bytes;
    l.sums = l.dz + (act ? round_up((size_t)q->M * l.lddz * 2, kWsAlign) : 0);
    l.part = l.sums + round_up((size_t)row_blocks(q->M, q->N) * q->N * sizeof(float), kWsAlign);
    l.products = plan_pair(px, pw);
    l.bytes = l.part + l.products.part;
    return GEMM_OK;
}

int run_linear_backward(bool bf16, const gemm_linear_backward_params *q, const uint16_t *dY, const uint16_t *X,
                        const uint16_t *W, const uint16_t *pre, uint16_t *dX, uint16_t *dW, uint16_t *dbias, void *ws,
                        size_t ws_bytes, void *stream)
{
    Product px, pw;
    BackwardLayout l;
    const int rc = check_linear_backward(q, px, pw, l);
    if (rc != GEMM_OK)
        return rc;
    const bool act = q->activation != GEMM_ACT_NONE;
    const int w_row = q->op_w ? q->K : q->N;
    if ((dX && (!ld_ok(q->ldw, w_row) || !ld_ok(q->lddx, q->K))) ||
        (dW && (!ld_ok(q->ldx, q->K) || !ld_ok(q->lddw, w_row))) || (act && !ld_ok(q->ldp, q->N)))
        return GEMM_ERR_INVALID_LAYOUT;
    if (missing(dY, q->M, q->N) || (act && missing(pre, q->M, q->N)) || (dX && missing(W, q->K, q->N)) ||
        (dW && missing(X, q->M, q->K)))
        return GEMM_ERR_NULL_PTR;
    if (!workspace_ok(ws, ws_bytes, l.bytes))
        return GEMM_ERR_WORKSPACE;
    const int dev = dgor::device_status();
    if (dev != GEMM_OK)
        return dev;
    hipStream_t s = (hipStream_t)stream;
    uint8_t *base = (uint8_t *)ws;
    const uint16_t *dZ = dY;
    const int blocks = row_blocks(q->M, q->N);
    float *sums = dbias && blocks != 1 ? (float *)(base + l.sums) : nullptr;
    px.bf16 = pw.bf16 = bf16;
    dZ = l.c.use(dX || dW ? l.copy_dy : -1, dZ, base);
    const uint16_t *Xs = l.c.use(dW ? l.copy_x : -1, X, base), *Ws = l.c.use(dX ? l.copy_w : -1, W, base);
    hipError_t err;
    if (q->M > 0 && q->N > 0 && ((act && (dX || dW)) || dbias)) {
        uint16_t *out = act && (dX || dW) ? (uint16_t *)(base + l.dz) : nullptr;
        err = dgor::launch_act_grad(q->M, q->N, dY, q->lddy, act ? pre : nullptr, q->ldp, out, l.lddz, q->activation,
                                    sums, blocks == 1 ? dbias : nullptr, l.c.marked(), bf16, s);
        if (out)
            dZ = out;
    } else {
        err = dgor::launch_repack(l.c.marked(), s);
    }
    // no rows: an empty sum, no workspace
    if (err == hipSuccess && dbias && blocks != 1 && q->N > 0)
        err = dgor::launch_sum_blocks(blocks, q->N, sums, dbias, bf16, s);
    if (err != hipSuccess)
        return GEMM_ERR_LAUNCH;
    if (dX) {
        px.A[0] = px.A[1] = dZ;
        px.B[0] = px.B[1] = Ws;
        px.e.Y = dX, px.e.ldy = q->lddx;
    }
    if (dW) {
        const bool t = q->op_w == GEMM_OP_T;
        pw.A[0] = pw.A[1] = t ? dZ : Xs;
        pw.B[0] = pw.B[1] = t ? Xs : dZ;
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
    p.A[0] = p.A[1] = c.use(copy[0], X, base);
    p.B[0] = c.use(copy[1], Wg, base), p.B[1] = c.use(copy[2], Wu, base);
    p.e.Y = H, p.e.ldy = q->ldh;
    p.e.pre = G, p.e.pre2 = U, p.e.ldp = q->ldp;
    const hipError_t err = dgor::launch_repack(c.marked(), s);
    return done(err == hipSuccess ? run_product(p, l, base + c.bytes, s) : err);
}

// Workspace of the gated backward pass: copies, dG and dU, then the partial
// sums of whichever product is running.
struct GatedBackwardLayout {
    Copies c;
    PairPlan products;
    int copy_x, copy_wg, copy_wu;
    int ldd;
    size_t dg, du, part, bytes;
};

int check_gated_backward(const gemm_gated_backward_params *q, Product &px, Product &pw, GatedBackwardLayout &l)
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    if (q->M < 0 || q->F < 0 || q->K < 0 || too_large(q->M, q->F) || too_large(q->M, q->K) || too_large(q->K, q->F))
        return GEMM_ERR_INVALID_DIM;
    if (!op_ok(q->op_w) || !ld_ok(q->lddh, q->F) || !ld_ok(q->ldp, q->F))
        return GEMM_ERR_INVALID_LAYOUT;
    if (!act_ok(q->activation))
        return GEMM_ERR_INVALID_ACTIVATION;
    l.ldd = (int)round_up((size_t)q->F, 8);
    const bool t = q->op_w == GEMM_OP_T;
    int ldx = q->ldx, ldw = q->ldw, ldu = q->ldw;
    px = input_gradient_product(q->M, q->F, q->K, q->op_w, l.ldd, ldw, 2);
    pw = weight_gradient_product(q->M, q->F, q->K, q->op_w, ldx, l.ldd, 2);
    const bool for_x = !few_rows(px) && worth_copies(px), for_w = worth_copies(pw);
    l.copy_x = for_w ? l.c.add(q->M, q->K, ldx) : -1;
    l.copy_wg = for_x ? l.c.add(t ? q->F : q->K, t ? q->K : q->F, ldw) : -1;
    l.copy_wu = for_x ? l.c.add(t ? q->F : q->K, t ? q->K : q->F, ldu) : -1;
    px.ldb = ldw;
    pw = weight_gradient_product(q->M, q->F, q->K, q->op_w, ldx, l.ldd, 2);
    px.units = l.c.units && (for_x || whole_units(t ? q->K : q->F, ldw));
    pw.units = l.c.units && (for_w || whole_units(q->K, ldx));
    const size_t d_bytes = round_up((size_t)q->M * l.ldd * 2, kWsAlign);
    l.dg = l.c.bytes;
    l.du = l.dg + d_bytes;
    l.part = l.du + d_bytes;
    l.products = plan_pair(px, pw);
    l.bytes = l.part + l.products.part;
    return GEMM_OK;
}

int run_gated_backward(bool bf16, const gemm_gated_backward_params *q, const uint16_t *dH, const uint16_t *X,
                       const uint16_t *Wg, const uint16_t *Wu, const uint16_t *G, const uint16_t *U, uint16_t *dX,
                       uint16_t *dWg, uint16_t *dWu, void *ws, size_t ws_bytes, void *stream)
{
    Product px, pw;
    GatedBackwardLayout l;
    const int rc = check_gated_backward(q, px, pw, l);
    if (rc != GEMM_OK)
        return rc;
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
    if (!workspace_ok(ws, ws_bytes, l.bytes))
        return GEMM_ERR_WORKSPACE;
    const int dev = dgor::device_status();
    if (dev != GEMM_OK)
        return dev;
    hipStream_t s = (hipStream_t)stream;
    uint8_t *base = (uint8_t *)ws;
    uint16_t *dG = (uint16_t *)(base + l.dg), *dU = (uint16_t *)(base + l.du);
    px.bf16 = pw.bf16 = bf16;
    const uint16_t *Xs = l.c.use(dWg ? l.copy_x : -1, X, base);
    const uint16_t *Gs = l.c.use(dX ? l.copy_wg : -1, Wg, base), *Us = l.c.use(dX ? l.copy_wu : -1, Wu, base);
    const hipError_t err = q->M > 0 && q->F > 0
                               ? dgor::launch_gate_grad(q->M, q->F, dH, q->lddh, G, U, q->ldp, dG, dU, l.ldd,
                                                        q->activation, l.c.marked(), bf16, s)
                               : dgor::launch_repack(l.c.marked(), s);
    if (err != hipSuccess)
        return GEMM_ERR_LAUNCH;
    if (dX) {
        px.A[0] = dG, px.A[1] = dU;
        px.B[0] = Gs, px.B[1] = Us;
        px.e.Y = dX, px.e.ldy = q->lddx;
    }
    if (dWg) {
        const bool t = q->op_w == GEMM_OP_T;
        pw.A[0] = t ? dG : Xs, pw.A[1] = t ? dU : Xs;
        pw.B[0] = t ? Xs : dG, pw.B[1] = t ? Xs : dU;
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
    const int rc = check_linear_backward(params, px, pw, l);
    if (rc == GEMM_OK)
        *bytes = l.bytes;
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
    const int rc = check_gated_backward(params, px, pw, l);
    if (rc == GEMM_OK)
        *bytes = l.bytes;
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
