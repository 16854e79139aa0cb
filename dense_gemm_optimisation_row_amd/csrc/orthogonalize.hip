// The orthogonalised update of a gradient by Newton-Schulz steps (declared in
// include/gemm.h).  With X the m x n matrix, m <= n (a taller one is turned round
// where it is read and written), a step is
//   A = X X^T,  P = a I + b A + c A A,  X <- P X.
// A and A A are symmetric: only the tiles on and below the diagonal are computed,
// each written to both places.
//
// Precision.  A step multiplies small singular values by a, five by 485, so what
// is rounded off X at the start grows by that against directions that grow less:
// operands rounded to 16 bits once leave errors of 2^-9 and more in the result.
// So each operand is two binary16 terms, hi + lo, and a product three on the matrix
// cores, hi hi + lo hi + hi lo (lo lo is below the terms' own error): 22 to 23
// bits at a third of the 16-bit rate, five times the FP32 one.  Terms are held at a
// power of two: the coefficients bound the singular values of each step on the
// host, so X, A and P have scales at which no entry overflows, and entries down to
// 2^-18 of the bound keep all bits, smaller ones an error of 2^-40 of it.  The Gram
// matrix alone would do for long rows (P's products applied to X once), but its
// rounding, 2^-24 of the largest eigenvalue, is a singular value of 2^-12.
//
// Bound by the matrix cores where the tiles fill the compute units.
#include <cmath>
#include <stdint.h>

#include "ring.h"
#include "ring_plan.h"

namespace dgor {
namespace {

using namespace ring;

struct OpHalf : Half16 {
    static __device__ __forceinline__ floatx4 mfma(halfx8 a, halfx8 b, floatx4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

enum Format { kF32, kF16, kBF16 };

__device__ __forceinline__ void load8_of(int fmt, const void *p, size_t at, int n, float (&f)[8])
{
    if (fmt == kF32)
        load8_f32((const float *)p + at, n, f);
    else if (fmt == kF16)
        unpack8<Half16>(load8_16((const uint16_t *)p + at, n), f);
    else
        unpack8<Brain16>(load8_16((const uint16_t *)p + at, n), f);
}
__device__ __forceinline__ void store8_of(int fmt, void *p, size_t at, int n, const float (&f)[8])
{
    if (fmt == kF32)
        store8_f32((float *)p + at, n, f);
    else
        store8_16((uint16_t *)p + at, n, fmt == kF16 ? pack8<Half16>(f) : pack8<Brain16>(f));
}

// Matrices in two terms: rows padded with zeros to whole units.
struct Pair {
    uint16_t *hi;
    long long term, matrix;   // elements from a value's higher term to its lower, and to the next matrix
    int ld;
    __device__ __forceinline__ void load8(long long m, int row, int col, float (&f)[8]) const
    {
        const uint16_t *p = hi + m * matrix + (size_t)row * ld + col;
        float lo[8];
        unpack8<Half16>(*reinterpret_cast<const u32x4 *>(p), f);
        unpack8<Half16>(*reinterpret_cast<const u32x4 *>(p + term), lo);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] += lo[e];
    }
    __device__ __forceinline__ void store8(long long m, int row, int col, const float (&f)[8]) const
    {
        uint16_t *p = hi + m * matrix + (size_t)row * ld + col;
        const u32x4 h = pack8<Half16>(f);
        float r[8];
        unpack8<Half16>(h, r);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r[e] = f[e] - r[e];
        *reinterpret_cast<u32x4 *>(p) = h;
        *reinterpret_cast<u32x4 *>(p + term) = pack8<Half16>(r);
    }
};

// ------------------------------------------------------------------ start --

// G as it is stored: rows x cols, at strides ld and `matrix`.
struct Source {
    const void *p;
    int rows, cols, ld;
    long long matrix;
    int fmt;
    __device__ __forceinline__ void load8(long long m, int row, int col, float (&f)[8]) const
    {
        load8_of(fmt, p, m * matrix + (size_t)row * ld + col, cols - col, f);
    }
};

// Adds 256 threads' doubles, in one order.
__device__ __forceinline__ double block_sum(double v, double *lds)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v += __shfl_xor(v, o, 64);
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// Sums of squares of each of `blocks` parts of each matrix, in FP64, which
// holds the square of any FP32.  Threads: 256 >> lg rows of 1 << lg units.
__global__ __launch_bounds__(256) void squares_kernel(Source g, int blocks, int lg, double *sums)
{
    __shared__ double lds[4];
    const long long m = blockIdx.x / blocks;
    const int part = (int)(blockIdx.x - m * blocks), across = 1 << lg, down = 256 >> lg;
    double v = 0;
    for (long long r = (long long)part * down + (threadIdx.x >> lg); r < g.rows; r += (long long)blocks * down)
        for (long long c = 8 * (threadIdx.x & (across - 1)); c < g.cols; c += 8 * across) {
            float f[8];
            g.load8(m, (int)r, (int)c, f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v += (double)f[e] * (double)f[e];
        }
    v = block_sum(v, lds);
    if (threadIdx.x == 0)
        sums[blockIdx.x] = v;
}

// X = G 2^s / (|G| + eps) in two terms; a block of 64 x 64 a workgroup, turned
// round through LDS where X is G's transpose.
__global__ __launch_bounds__(256) void start_kernel(Source g, Pair x, const double *sums, int blocks, double eps,
                                                    double by, int across, int per, bool turned)
{
    __shared__ double lds[4];
    __shared__ float tile[64][65];
    const long long m = blockIdx.x / per;
    const int id = (int)(blockIdx.x - m * per), r0 = 64 * (id / across), c0 = 64 * (id % across);
    const double v = block_sum((int)threadIdx.x < blocks ? sums[m * blocks + threadIdx.x] : 0.0, lds);
    const double factor = by / (sqrt(v) + eps);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int r = (int)(threadIdx.x >> 3) + 32 * t, c = 8 * (int)(threadIdx.x & 7);
        float f[8] = {};
        if (r0 + r < g.rows && c0 + c < g.cols) {
            g.load8(m, r0 + r, c0 + c, f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = c0 + c + e < g.cols ? (float)(f[e] * factor) : 0.f;   // (zeros, whatever the factor)
            if (!turned)
                x.store8(m, r0 + r, c0 + c, f);
        }
        if (turned)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                tile[r][c + e] = f[e];
    }
    if (!turned)
        return;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int c = (int)(threadIdx.x >> 3) + 32 * t, r = 8 * (int)(threadIdx.x & 7);
        if (c0 + c < g.cols && r0 + r < g.rows) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = tile[r + e][c];
            x.store8(m, c0 + c, r0 + r, f);
        }
    }
}

// --------------------------------------------------------------- products --

// What becomes of a product's sums: alpha sum, or (polynomial) alpha sum + beta A
// and the diagonal on it, in two terms, or (out) rounded to the result's format,
// its transpose where `turned`.
struct Finish {
    bool polynomial;
    float alpha, beta, diagonal;
    Pair with;             // A, symmetric
    Pair to;
    void *out;             // null: to `to`
    long long out_matrix;
    int out_ld, fmt;
    bool turned;

    __device__ __forceinline__ void value(long long m, int row, int col, float (&v)[8]) const
    {
        if (polynomial) {
            float a[8];
            with.load8(m, row, col, a);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = __builtin_fmaf(alpha, v[e], beta * a[e]) + (row == col + e ? diagonal : 0.f);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] *= alpha;
        }
    }
    // Eight neighbouring elements of a row of the result, n of them inside it.  (Of
    // the symmetric results also the ones of a column: they are the same.)
    __device__ __forceinline__ void put(long long m, int row, int col, int n, float (&v)[8]) const
    {
        value(m, row, col, v);
        if (out)
            store8_of(fmt, out, m * out_matrix + (size_t)row * out_ld + col, n, v);
        else
            to.store8(m, row, col, v);
    }
};

// The tile of a symmetric result that workgroup `id` of `all` computes: row by row
// of the lower triangle, those of one XCD (id % 8) next to each other.
__device__ __forceinline__ void triangle_tile(int id, int all, int &tm, int &tn)
{
    const int per = all >> 3, rem = all & 7, xcd = id & 7;
    const int l = xcd * per + min(xcd, rem) + (id >> 3);
    int r = (int)((sqrtf(8.f * (float)l + 1.f) - 1.f) * 0.5f);
    while ((long long)(r + 1) * (r + 2) / 2 <= l)
        ++r;
    while ((long long)r * (r + 1) / 2 > l)
        --r;
    tm = r;
    tn = l - r * (r + 1) / 2;
}

struct Batch {
    long long a, b;   // elements from a matrix's operands to the next one's
    int per;          // tiles of a matrix
};

template <int BM, int BN, bool TB, bool SYM>
__global__ __launch_bounds__(256) void newton_schulz_kernel(Product p, Batch batch, Finish f)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[ring_bytes(BM, BN, false)];
    constexpr int HM = BM / 2, HN = BN / 2, FA = HM / 16, FB = HN / 16;
    const int m = (int)blockIdx.x / batch.per, id = (int)blockIdx.x - m * batch.per, part = (int)blockIdx.y;
    int tm, tn;
    if (SYM)
        triangle_tile(id, batch.per, tm, tn);
    else
        dgor_tile_of_block(id, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    p.A.p += m * batch.a;
    p.B.p += m * batch.b;
    floatx4 acc[FA][FB];
    ring_sum<OpHalf, BM, BN, false, TB, false>(p, lds, tm, tn, 0, part, acc);

    // 32 rows at a time through the wavefront's own part of LDS
    constexpr int ROW = HN + 4, LANES = HN / 8, STEP = 64 / LANES;
    static_assert(4 * 32 * ROW * 4 <= ring_bytes(BM, BN, false), "the epilogue uses the ring's LDS");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    float *w = reinterpret_cast<float *>(lds) + wave * 32 * ROW;
    const int first = tm * BM + (wave >> 1) * HM, left = tn * BN + (wave & 1) * HN;
    const bool along = p.splits > 1 || !f.turned, across = p.splits <= 1 && (f.turned || (SYM && tm != tn));
#pragma unroll 1
    for (int round = 0; round < FA / 2; ++round) {
        stage_rows(acc, round, w, ROW, lane);
        const int top = first + 32 * round;
        if (along) {
            const int c = 8 * (lane % LANES), col = left + c;
#pragma unroll 1
            for (int r = lane / LANES; r < 32; r += STEP) {
                const int row = top + r;
                if (row >= p.M || col >= p.N)
                    break;
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = w[r * ROW + c + e];
                if (p.splits > 1)
                    store8_f32(p.part + ((long long)m * p.splits + part) * part_size(p) +
                                   (size_t)row * part_stride(p) + col, 8, v);
                else
                    f.put(m, row, col, p.N - col, v);
            }
        }
        if (across) {   // four lanes a column: 64 bytes of 16-bit results
            const int r = 8 * (lane & 3), row = top + r;
#pragma unroll 1
            for (int c = lane >> 2; c < HN; c += 16) {
                const int col = left + c;
                if (row >= p.M || col >= p.N)
                    break;
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = w[(r + e) * ROW + c];
                f.put(m, col, row, p.M - row, v);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// Adds the parts of split sums: a 64 x 64 block a workgroup.
template <bool SYM>
__global__ __launch_bounds__(256) void newton_schulz_join_kernel(Product p, Batch batch, Finish f)
{
    __shared__ float tile[64][68];
    const int m = (int)blockIdx.x / batch.per, id = (int)blockIdx.x - m * batch.per;
    int tm, tn;
    if (SYM)
        triangle_tile(id, batch.per, tm, tn);
    else
        dgor_tile_of_block(id, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    const bool across = f.turned || (SYM && tm != tn);
    const int r0 = 64 * tm, c0 = 64 * tn;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int r = (int)(threadIdx.x >> 3) + 32 * t, c = 8 * (int)(threadIdx.x & 7);
        float v[8] = {};
        if (r0 + r < p.M && c0 + c < p.N) {
            const float *from = p.part + (long long)m * p.splits * part_size(p) + (size_t)(r0 + r) * part_stride(p) + c0 + c;
            load8_f32(from, 8, v);
            for (int s = 1; s < p.splits; ++s) {
                float u[8];
                load8_f32(from + s * part_size(p), 8, u);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] += u[e];
            }
        }
        if (across)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                tile[r][c + e] = v[e];
        if (!f.turned && r0 + r < p.M && c0 + c < p.N)
            f.put(m, r0 + r, c0 + c, p.N - c0 - c, v);
    }
    if (!across)
        return;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int c = (int)(threadIdx.x >> 3) + 32 * t, r = 8 * (int)(threadIdx.x & 7);
        if (r0 + r < p.M && c0 + c < p.N) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = tile[r + e][c];
            f.put(m, c0 + c, r0 + r, p.M - r0 - r, v);
        }
    }
}

// ------------------------------------------------------------------- host --

constexpr size_t kWsAlign = 256;
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
// A launch holds fewer than 2^32 threads.
constexpr long long kMostGroups = 1 << 24;

// The three products of a step.
enum Which { kGram, kPolynomial, kUpdate };
struct Way {
    RingTile tile;
    int splits, chunk;
};

long long tiles_of(Which which, int m, int n, int bm, int bn)
{
    const long long down = ceil_div(m, bm);
    return which == kUpdate ? down * ceil_div(n, bn) : down * (down + 1) / 2;
}

Product product_of(Which which, int m, int n)
{
    Product p{};
    p.M = m, p.N = which == kUpdate ? n : m, p.K = which == kGram ? n : m;
    p.trans_b = which != kUpdate;
    p.units = true;
    p.nseg = p.terms = 3;
    p.nbatch = p.splits = 1;
    p.A.low = 1, p.B.low = 2;
    p.group_m = 4;
    return p;
}

// The tile and the split of the sum by the rings' times (ring_plan.h).
Way choose(Which which, int m, int n, int batch)
{
    const Product p = product_of(which, m, n);
    const int stages = product_stages(p);
    Way w{kRing64, 1, 0};
    double best = 0;
    bool any = false;
    for (const RingCost &c : kRings) {
        const int bm = ring_tile_m(c.tile), bn = ring_tile_n(c.tile);
        if (which != kUpdate && bm != bn)
            continue;
        const long long groups = batch * tiles_of(which, m, n, bm, bn);
        for (int parts : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
            if (parts > 1 && (2 * parts > stages || groups * parts > 512 * c.share))
                break;
            if (groups * parts >= kMostGroups)
                break;
            const RingTimes t = times(p, c, parts);
            const long long all = groups * parts, rounds = all / (256 * c.share), rest = all % (256 * c.share);
            double us = rounds * t.full + (rest == 0 ? 0.0 : rest <= 256 ? t.alone : t.full);
            if (parts > 1)
                us += kJoinLaunch + (which == kUpdate ? 8.0 : 4.0) * parts * batch * p.M * p.N / kJoinBytes;
            if (!any || us < best) {
                any = true, best = us, w.tile = c.tile;
                w.chunk = parts > 1 ? ceil_div(stages, parts) : 0;
                w.splits = parts > 1 ? ceil_div(stages, w.chunk) : 1;
            }
        }
    }
    return w;
}

// Bounds of a step: of X's singular values, and of the polynomial on X X^T's
// eigenvalues.  |a s + b s^3 + c s^5| and |a + b t + c t^2| over [0, r] and [0,
// r^2]: at the ends and where the derivative is zero.
double grown(double a, double b, double c, double r)
{
    const auto f = [&](double s) { return std::fabs(s * (a + s * s * (b + s * s * c))); };
    double most = f(r);
    const auto at = [&](double t) {   // a zero of a + 3 b t + 5 c t^2, t = s^2
        if (t > 0 && t < r * r)
            most = std::fmax(most, f(std::sqrt(t)));
    };
    if (c != 0) {
        const double d = 9 * b * b - 20 * a * c;
        if (d >= 0) {
            at((-3 * b + std::sqrt(d)) / (10 * c));
            at((-3 * b - std::sqrt(d)) / (10 * c));
        }
    } else if (b != 0) {
        at(-a / (3 * b));
    }
    return most;
}
double multiplied(double a, double b, double c, double r)
{
    const double t = r * r;
    const auto f = [&](double v) { return std::fabs(a + v * (b + v * c)); };
    double most = std::fmax(f(0), f(t));
    if (c != 0 && -b / (2 * c) > 0 && -b / (2 * c) < t)
        most = std::fmax(most, f(-b / (2 * c)));
    return most;
}
// The power of two at which values of at most `most` stay binary16: the rounding
// of the sums is far below what 60000 leaves to 65504.
int exponent_for(double most)
{
    int e = 0;
    std::frexp(60000.0 / std::fmax(most, 1.0), &e);   // 60000 / most in [2^(e - 1), 2^e)
    return e - 1;
}

struct Step {
    double a, b, c;
    int x, gram, poly;   // exponents of X, A and P
};

struct Layout {
    int m, n, ldx, lda;
    bool turned_in, turned_out;
    int blocks, lg;          // of the sums of squares
    Way way[3];
    Step step[GEMM_MAX_STEPS];
    size_t sums, x[2], gram, poly, part, bytes;   // offsets, and the whole size
};

bool ld_ok(int ld, int row) { return ld >= (row > 1 ? row : 1); }

int lay_out(const gemm_orthogonalize_params *q, Layout &l)
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    constexpr int LONGEST = (1 << 22) - 8;   // the rings' strides
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
        if (!(p <= 256) || !(next <= 256))
            return GEMM_ERR_INVALID_COEFFICIENTS;
        s.x = exponent_for(r), s.gram = exponent_for(r * r), s.poly = exponent_for(p);
        r = next;
    }
    if (q->batch == 0 || q->M == 0 || q->N == 0)
        return GEMM_OK;
    const bool tall = q->M > q->N;
    l.m = tall ? q->N : q->M, l.n = tall ? q->M : q->N;
    l.turned_in = tall != (q->op_g == GEMM_OP_T), l.turned_out = tall != (q->op_o == GEMM_OP_T);
    l.ldx = (int)round_up((size_t)l.n, 8), l.lda = (int)round_up((size_t)l.m, 8);
    for (int i = 0; i < 3; ++i) {
        l.way[i] = choose((Which)i, l.m, l.n, q->batch);
        const Way &w = l.way[i];
        if (q->batch * tiles_of((Which)i, l.m, l.n, ring_tile_m(w.tile), ring_tile_n(w.tile)) * w.splits >= kMostGroups)
            return GEMM_ERR_INVALID_DIM;
    }
    if (q->batch * (long long)ceil_div(l.m, 64) * ceil_div(l.n, 64) >= kMostGroups)
        return GEMM_ERR_INVALID_DIM;
    // parts of at least 8192 elements, at most 256 (start_kernel's threads)
    const long long parts = ((long long)l.m * l.n + 8191) / 8192;
    l.blocks = (int)(parts < 256 ? parts : 256);
    if (q->batch * (long long)l.blocks >= kMostGroups)
        return GEMM_ERR_INVALID_DIM;
    const int cols = l.turned_in ? l.m : l.n;
    while (l.lg < 8 && (8 << l.lg) < cols)
        ++l.lg;
    const auto take = [&](size_t bytes) {
        const size_t at = l.bytes;
        l.bytes += round_up(bytes, kWsAlign);
        return at;
    };
    const size_t b = (size_t)q->batch, x = 4 * b * l.m * l.ldx, a = 4 * b * l.m * l.lda;   // two terms of two bytes
    l.sums = take(sizeof(double) * b * l.blocks);
    l.x[0] = take(x);
    l.x[1] = q->steps > 1 ? take(x) : l.x[0];
    l.gram = take(a);
    l.poly = take(a);
    size_t part = 0;
    for (int i = 0; i < 3; ++i)
        if (l.way[i].splits > 1) {
            const size_t v = sizeof(float) * b * l.way[i].splits * part_size(product_of((Which)i, l.m, l.n));
            part = v > part ? v : part;
        }
    l.part = take(part);
    return GEMM_OK;
}

template <int BM, int BN>
void launch_as(Which which, const Product &p, const Batch &b, const Finish &f, const dim3 &grid, hipStream_t s)
{
    if (which == kUpdate)
        hipLaunchKernelGGL((newton_schulz_kernel<BM, BN, false, false>), grid, dim3(256), 0, s, p, b, f);
    else if constexpr (BM == BN)
        hipLaunchKernelGGL((newton_schulz_kernel<BM, BN, true, true>), grid, dim3(256), 0, s, p, b, f);
}

hipError_t launch(Which which, Product p, const Way &w, Batch b, const Finish &f, int batch, hipStream_t s)
{
    const int bm = ring_tile_m(w.tile), bn = ring_tile_n(w.tile);
    p.splits = w.splits, p.chunk = w.chunk;
    p.tiles_m = ceil_div(p.M, bm), p.tiles_n = ceil_div(p.N, bn);
    b.per = (int)tiles_of(which, p.M, p.N, bm, bn);
    const dim3 grid((unsigned)(batch * b.per), (unsigned)w.splits);
    switch (w.tile) {
    case kRing256: launch_as<256, 256>(which, p, b, f, grid, s); break;
    case kRing256x128: launch_as<256, 128>(which, p, b, f, grid, s); break;
    case kRing128: launch_as<128, 128>(which, p, b, f, grid, s); break;
    case kRing128x64: launch_as<128, 64>(which, p, b, f, grid, s); break;
    case kRing64: launch_as<64, 64>(which, p, b, f, grid, s); break;
    }
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || w.splits <= 1)
        return err;
    p.tiles_m = ceil_div(p.M, 64), p.tiles_n = ceil_div(p.N, 64);
    b.per = (int)tiles_of(which, p.M, p.N, 64, 64);
    const dim3 blocks((unsigned)(batch * b.per));
    if (which == kUpdate)
        hipLaunchKernelGGL((newton_schulz_join_kernel<false>), blocks, dim3(256), 0, s, p, b, f);
    else
        hipLaunchKernelGGL((newton_schulz_join_kernel<true>), blocks, dim3(256), 0, s, p, b, f);
    return hipGetLastError();
}

int run(int fmt, const gemm_orthogonalize_params *q, const void *G, void *O, void *ws, size_t ws_bytes, void *stream)
{
    Layout l;
    const int rc = lay_out(q, l);
    if (rc != GEMM_OK)
        return rc;
    if (q->batch == 0 || q->M == 0 || q->N == 0)
        return GEMM_OK;
    if (!G || !O)
        return GEMM_ERR_NULL_PTR;
    if (!ws || ws_bytes < l.bytes || ((uintptr_t)ws & (kWsAlign - 1)) != 0)
        return GEMM_ERR_WORKSPACE;
    const int dev = device_status();
    if (dev != GEMM_OK)
        return dev;
    hipStream_t s = (hipStream_t)stream;
    uint8_t *base = (uint8_t *)ws;
    const int batch = q->batch;
    const auto pair = [&](size_t at, int ld) {
        const long long size = (long long)l.m * ld;
        return Pair{(uint16_t *)(base + at), batch * size, size, ld};
    };
    const Pair x[2] = {pair(l.x[0], l.ldx), pair(l.x[1], l.ldx)}, gram = pair(l.gram, l.lda), poly = pair(l.poly, l.lda);

    const bool t = q->op_g == GEMM_OP_T;
    const Source g{G, t ? q->N : q->M, t ? q->M : q->N, q->ldg, batch > 1 ? q->stride_g : 0, fmt};
    double *sums = (double *)(base + l.sums);
    hipLaunchKernelGGL(squares_kernel, dim3((unsigned)(batch * l.blocks)), dim3(256), 0, s, g, l.blocks, l.lg, sums);
    const int across = ceil_div(g.cols, 64), per = across * ceil_div(g.rows, 64);
    hipLaunchKernelGGL(start_kernel, dim3((unsigned)(batch * per)), dim3(256), 0, s, g, x[0], sums, l.blocks, q->eps,
                       std::ldexp(1.0, l.step[0].x), across, per, l.turned_in);
    hipError_t err = hipGetLastError();

    const auto of = [&](Which which, const Pair &a, const Pair &b) {
        Product p = product_of(which, l.m, l.n);
        p.A = {a.hi, 0, 2 * a.term, 1};
        p.B = {b.hi, 0, 2 * b.term, 2};
        p.lda = a.ld, p.ldb = b.ld;
        p.part = (float *)(base + l.part);
        return p;
    };
    for (int i = 0; i < q->steps && err == hipSuccess; ++i) {
        const Step &k = l.step[i];
        const Pair &now = x[i & 1], &next = x[(i + 1) & 1];
        Finish f{};
        f.alpha = (float)std::ldexp(1.0, k.gram - 2 * k.x);
        f.to = gram;
        err = launch(kGram, of(kGram, now, now), l.way[kGram], {now.matrix, now.matrix, 0}, f, batch, s);
        if (err != hipSuccess)
            break;
        f.polynomial = true;
        f.alpha = (float)std::ldexp(k.c, k.poly - 2 * k.gram);
        f.beta = (float)std::ldexp(k.b, k.poly - k.gram);
        f.diagonal = (float)std::ldexp(k.a, k.poly);
        f.with = gram, f.to = poly;
        err = launch(kPolynomial, of(kPolynomial, gram, gram), l.way[kPolynomial], {gram.matrix, gram.matrix, 0}, f, batch, s);
        if (err != hipSuccess)
            break;
        f = Finish{};
        if (i + 1 < q->steps) {
            f.alpha = (float)std::ldexp(1.0, l.step[i + 1].x - k.poly - k.x);
            f.to = next;
        } else {
            f.alpha = (float)std::ldexp(q->scale, -k.poly - k.x);
            f.out = O, f.out_ld = q->ldo, f.out_matrix = batch > 1 ? q->stride_o : 0;
            f.fmt = fmt, f.turned = l.turned_out;
        }
        err = launch(kUpdate, of(kUpdate, poly, now), l.way[kUpdate], {poly.matrix, now.matrix, 0}, f, batch, s);
    }
    return err == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace
}  // namespace dgor

extern "C" {

int gemm_orthogonalize_workspace(const gemm_orthogonalize_params *params, size_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_NULL_PTR;
    dgor::Layout l;
    const int rc = dgor::lay_out(params, l);
    if (rc == GEMM_OK)
        *bytes = l.bytes;
    return rc;
}
int gemm_orthogonalize_f32(const gemm_orthogonalize_params *params, const float *G, float *O, void *workspace,
                           size_t workspace_bytes, void *stream)
{
    return dgor::run(dgor::kF32, params, G, O, workspace, workspace_bytes, stream);
}
int gemm_orthogonalize_f16(const gemm_orthogonalize_params *params, const uint16_t *G, uint16_t *O, void *workspace,
                           size_t workspace_bytes, void *stream)
{
    return dgor::run(dgor::kF16, params, G, O, workspace, workspace_bytes, stream);
}
int gemm_orthogonalize_bf16(const gemm_orthogonalize_params *params, const uint16_t *G, uint16_t *O, void *workspace,
                            size_t workspace_bytes, void *stream)
{
    return dgor::run(dgor::kBF16, params, G, O, workspace, workspace_bytes, stream);
}

}  // extern "C"
