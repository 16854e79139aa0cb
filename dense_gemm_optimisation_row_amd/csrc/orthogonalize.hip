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
// So each operand is two binary16 terms, hi + lo, which hold a value to 2^-23 (FP32
// would to 2^-24), and a product three on the matrix cores, hi hi + lo hi + hi lo, at a
// third of the 16-bit rate, five times the FP32 one; lo lo, at most 2^-22 of a product,
// is added where the sums are of few.  Over 160 sizes the result's error is 0.61 times
// that of FP32 products at the median and 1.03 times at most, up to 1.23 times where the
// directions fall off as 1 / k; a third term would take twice the products.  Terms are
// held at a power of two: the coefficients bound the singular values of each step on the
// host, so X, A and P have scales at which no entry overflows, and entries down to
// 2^-16 of the bound keep all bits, smaller ones are off by at most 2^-39 of it.  The Gram
// matrix alone would do for long rows (P's products applied to X once), but its
// rounding, 2^-24 of the largest eigenvalue, is a singular value of 2^-12.
//
// Bound by the matrix cores where the tiles fill the compute units.
#include <cstddef>
#include <stdint.h>
#include <type_traits>

#include "orthogonalize.h"
#include "ring.h"

namespace dgor {
namespace {

using namespace newton_schulz;
using namespace ring;

typedef _Float16 halfx4 __attribute__((ext_vector_type(4)));

// Matrices in two terms.  A row is groups of 32 columns, each 64 bytes of higher
// terms and then 64 of lower ones, so that what a 32-deep stage takes of a row is
// one whole line of 128 bytes: a compute unit takes about as many pieces a
// microsecond whatever their size, and from two matrices, 64 bytes at a time, the
// 64 x 64 tile took 17 us for 777 x 1033 by its transpose.  Rows are padded
// with zeros to whole units of eight.
struct Pair {
    uint16_t *p;
    long long matrix;   // elements from a matrix to the next
    int ld;
    __device__ __forceinline__ uint16_t *at(long long m, int row, int col) const
    {
        return p + m * matrix + (size_t)row * ld + 2 * (col & ~31) + (col & 31);
    }
    __device__ __forceinline__ void load8(long long m, int row, int col, float (&f)[8]) const
    {
        const uint16_t *q = at(m, row, col);
        float lo[8];
        unpack8<Half16>(*reinterpret_cast<const u32x4 *>(q), f);
        unpack8<Half16>(*reinterpret_cast<const u32x4 *>(q + 32), lo);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] += lo[e];
    }
    __device__ __forceinline__ void store8(long long m, int row, int col, const float (&f)[8]) const
    {
        uint16_t *q = at(m, row, col);
        const u32x4 h = pack8<Half16>(f);
        float r[8];
        unpack8<Half16>(h, r);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            r[e] = f[e] - r[e];
        *reinterpret_cast<u32x4 *>(q) = h;
        *reinterpret_cast<u32x4 *>(q + 32) = pack8<Half16>(r);
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

// What G is multiplied by, `by` / (|G| + eps), from its sum of squares, which is zero
// for zeros alone: these stay zeros, whatever eps.
__device__ __forceinline__ double factor_of(double by, double squares, double eps)
{
    return squares == 0 ? 0 : by / (sqrt(squares) + eps);
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
    double v = 0;
    for (int i = threadIdx.x; i < blocks; i += 256)
        v += sums[m * blocks + i];
    v = block_sum(v, lds);
    const double factor = factor_of(by, v, eps);
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
    // [1]: what is left of the coefficient after its rounding to FP32.  Where the
    // singular values are near 1, a + b + c is far below a and b, and so are P's
    // entries: their terms' roundings would weigh 5 to 7 times as much in them.
    float alpha[2], beta[2], diagonal[2];
    Pair with;             // A, symmetric
    Pair to;
    void *out;             // null: to `to`
    long long out_matrix;
    int out_ld, fmt;
    bool turned;

    // Eight neighbouring elements of a row: their value from the sums v and, of the
    // polynomial, A's elements a (of the symmetric results a column's are a row's).
    __device__ __forceinline__ void value(int row, int col, float (&v)[8], const float (&a)[8]) const
    {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (polynomial) {
                // the large terms cancel first, in the FMAs, which round once
                const bool on = row == col + e;
                const float rest = __builtin_fmaf(alpha[1], v[e], __builtin_fmaf(beta[1], a[e], on ? diagonal[1] : 0.f));
                v[e] = __builtin_fmaf(alpha[0], v[e], __builtin_fmaf(beta[0], a[e], on ? diagonal[0] : 0.f)) + rest;
            } else {
                v[e] *= alpha[0];
            }
    }
    // n of them inside the result
    __device__ __forceinline__ void store(long long m, int row, int col, int n, const float (&v)[8]) const
    {
        if (out)
            store8_of(fmt, out, m * out_matrix + (size_t)row * out_ld + col, n, v);
        else
            to.store8(m, row, col, v);
    }
};

// One product of matrices in two terms: A, M x K, by B, N x K (TB) or K x N.
struct Operands {
    int M, N, K;
    Pair a, b;
};

// The 32-deep stages of all tiles of all matrices, dealt to the workgroups: the
// first `whole` tiles a tile at a time, in full rounds, in which the workgroups of an
// XCD read the same panels at the same time; the others' stages in runs of `run`,
// one run a workgroup.  A tile in several runs is left in FP32 in their slabs, two a
// workgroup (the tile that its run begins in, and the one that it ends in), and
// joined by another launch.
struct Work {
    int tiles, per, stages;   // tiles of all matrices and of one; stages of a tile
    int tiles_m, tiles_n;     // of one matrix's result
    int groups, whole, run;
    float *slabs;
    // slab of a tile that begins at stage `begin` of the runs' stages, in run w
    __device__ __forceinline__ size_t slab(int w, long long begin, int size) const
    {
        return (size_t)(2 * w + (begin >= (long long)w * run ? 1 : 0)) * size;
    }
};

// Tile `id` of a matrix: all of them, or (symmetric) those on and below the
// diagonal, row by row.
template <bool SYM>
__device__ __forceinline__ void tile_of(const Work &w, int id, int &tm, int &tn)
{
    if (SYM) {
        int r = (int)((sqrtf(8.f * (float)id + 1.f) - 1.f) * 0.5f);
        while ((long long)(r + 1) * (r + 2) / 2 <= id)
            ++r;
        while ((long long)r * (r + 1) / 2 > id)
            --r;
        tm = r;
        tn = id - (int)((long long)r * (r + 1) / 2);
    } else {
        // groups of four tile rows, column by column: neighbours share panels
        const int span = 4 * w.tiles_n, group = id / span, in = id - group * span, first = 4 * group;
        const int rows = min(w.tiles_m - first, 4);
        tm = first + in % rows;
        tn = in / rows;
    }
}

// The tile's main loop: 32-deep stages of both terms of both operands, loaded
// straight into a ring of NB LDS buffers, the fragments of the next stage read
// and the loads of the stage NB further issued between the MFMAs.  A block of 16 x
// 16 outputs takes three MFMAs from four fragments, where a loop over the three
// products would read six and load each operand's higher term twice.
//
// A stage buffer: A, then B.  Rows along k (A, and B as N x K): eight units of 16
// bytes a row, higher terms and then lower ones, unit c of row r at 8 r + (c ^
// ((r >> 1) & 7)).  B as K x N: two halves of the tile's columns, each 32 k rows of
// W = HN / 4 units, unit u of row k at W k + (u ^ x(k)), x as in ring.h.
//
// Before stage t: this wavefront's loads of stage t + 1 and its reads of stage t
// have returned, then a barrier.  So all of stage t + 1 has landed, and nobody
// still reads stage t's buffer, which the loads of stage t + NB refill.
template <int BM, int BN>
constexpr int stage_bytes() { return (BM + BN) * 32 * 2 * 2; }

// A wavefront's loads of a stage: of rows along k eight a load, LPA of A's and (B as N x
// K) LPB of B's; of B as K x N 64 / W k rows a load, of one half of the tile's columns.
template <int BM, int BN, bool TB>
struct StageLoads {
    static constexpr int BK = 32, HN = BN / 2, W = HN / 4;
    static constexpr int LPA = BM / 32, LPB = BN / 32, LOADS = LPA + LPB;
    static constexpr int HALF_B = HN * 128, B_AT = BM * 128;
    uint32_t a_off[2], b_off[TB ? 2 : LPB], a_rows, b_rows, at_a, at_b;
    int kc[2], lda, ldb, a_left, b_left, k_left;
    size_t b_step;   // elements from a k to the next
    const uint16_t *ap, *bp;
    // of tile (m0, n0) of matrix m, from stage s0; what is past k `end` reads as zero
    __device__ __forceinline__ StageLoads(const Operands &p, long long m, int m0, int n0, int s0, int end, int lane,
                                          int wave)
        : lda(p.a.ld), ldb(p.b.ld), a_left(p.M - m0), k_left(end - BK * s0)
    {
        const int lhalf = wave >> 1;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            // unit (lane % 8) of row lane / 8 holds k's unit `unit` & 3 of the term unit / 4
            const int unit = (lane & 7) ^ ((4 * q + (lane >> 4)) & 7);
            kc[q] = 8 * (unit & 3);
            a_off[q] = (uint32_t)((8 * (LPA * wave + q) + (lane >> 3)) * lda + 8 * unit) * 2u;
            if (TB)
                b_off[q] = (uint32_t)((8 * (LPB * wave + q) + (lane >> 3)) * ldb + 8 * unit) * 2u;
        }
        a_rows = (uint32_t)(16 * lda) * 2u, b_rows = (uint32_t)(16 * ldb) * 2u;
        const int bcol = TB ? n0 : n0 + HN * lhalf;
        b_left = p.N - bcol;
        if (!TB)
#pragma unroll
            for (int q = 0; q < LPB; ++q) {
                const int k = (64 / W) * (LPB * (wave & 1) + q) + lane / W;
                const int u = (lane % W) ^ row_swizzle<(W < 16 ? W : 16)>(k);
                b_off[TB ? 0 : q] = 32 * (u >> 3) + 8 * (u & 3) < b_left ? (uint32_t)(k * ldb + 8 * u) * 2u : kOutside;
            }
        b_step = TB ? 2 : (size_t)ldb;
        ap = p.a.p + m * p.a.matrix + (size_t)m0 * lda + (size_t)(2 * BK) * s0;
        bp = p.b.p + m * p.b.matrix + (TB ? (size_t)bcol * ldb : (size_t)(2 * bcol)) + BK * s0 * b_step;
        at_a = (uint32_t)(LPA * wave * 1024);
        at_b = (uint32_t)(B_AT + (TB ? LPB * wave * 1024 : lhalf * HALF_B + LPB * (wave & 1) * 1024));
    }
    struct Stage {
        intx4 a, b;
        int k_left;
    };
    __device__ __forceinline__ Stage next()
    {
        Stage L;
        L.k_left = k_left;
        L.a = rsrc_words(ap, 0);
        L.b = rsrc_words(bp, 0);
        L.a.z = k_left <= 0 ? 0 : (a_left >= BM ? 0x7fffffff : (a_left - 1) * lda * 2 + 128);
        if (TB)
            L.b.z = k_left <= 0 ? 0 : (b_left >= BN ? 0x7fffffff : (b_left - 1) * ldb * 2 + 128);
        else
            L.b.z = k_left >= BK || b_left <= 0 ? 0x7fffffff
                                                : (k_left <= 0 ? 0 : (k_left - 1) * ldb * 2 + 4 * ((b_left + 31) & ~31));
        ap += 2 * BK;
        bp += BK * b_step;
        k_left -= BK;
        return L;
    }
    // load i of a stage, into the buffer at the LDS address `to`
    __device__ __forceinline__ void load(const Stage &L, uint32_t to, int i) const
    {
        if (i < LPA)
            load_to_lds(L.a, to + at_a + (uint32_t)(i * 1024),
                        kc[i & 1] >= L.k_left ? kOutside : a_off[i & 1] + (uint32_t)(i >> 1) * a_rows);
        else if (TB)
            load_to_lds(L.b, to + at_b + (uint32_t)((i - LPA) * 1024),
                        kc[i & 1] >= L.k_left ? kOutside : b_off[(i - LPA) & 1] + (uint32_t)((i - LPA) >> 1) * b_rows);
        else
            load_to_lds(L.b, to + at_b + (uint32_t)((i - LPA) * 1024), b_off[TB ? 0 : i - LPA]);
    }
    static_assert(LPA % 2 == 0 && LPB % 2 == 0, "");
};

// Where a lane's fragments begin in a stage buffer.  Lane (g, s) = (lane / 16, lane %
// 16): k 8 g .. 8 g + 7 of row s of A's block and column s of B's.
template <int BM, int BN, bool TB>
struct StageLanes {
    static constexpr int HM = BM / 2, HN = BN / 2, W = HN / 4;
    static constexpr int UNITS = HN / 16 < 4 ? HN / 16 : 4;   // B's blocks from the fifth on are sixteen units on
    uint32_t a, b, b_unit[TB ? 1 : UNITS];   // b_unit: of the higher terms; the lower ones are four units on
    __device__ __forceinline__ StageLanes(int lane, int wave)
    {
        const int s16 = lane & 15, g = lane >> 4, kr = 8 * g + (s16 >> 2);
        const uint32_t row = (uint32_t)(s16 * 128) | (uint32_t)((g ^ ((s16 >> 1) & 7)) * 16);
        a = row + (uint32_t)((wave >> 1) * HM * 128);
        b = (uint32_t)(BM * 128) + (TB ? row + (uint32_t)((wave & 1) * HN * 128)
                                       : (uint32_t)(kr * (W * 16) + 8 * (s16 & 1) + (wave & 1) * HN * 128));
        if (!TB)
#pragma unroll
            for (int j = 0; j < UNITS; ++j)
                b_unit[TB ? 0 : j] = (uint32_t)(
                    ((8 * (j >> 1) + 2 * (j & 1) + ((s16 & 3) >> 1)) ^ row_swizzle<(W < 16 ? W : 16)>(kr)) * 16);
    }
    // term of A's block i and B's block j, of the buffer at byte `at`
    __device__ __forceinline__ halfx8 read_a(const uint8_t *lds, uint32_t at, int i, int term) const
    {
        return *reinterpret_cast<const halfx8 *>(lds + ((a ^ (uint32_t)(64 * term)) + (at + (uint32_t)(i * 2048))));
    }
    __device__ __forceinline__ halfx8 read_b(const uint8_t *lds, uint32_t at, int j, int term) const
    {
        if (TB)
            return *reinterpret_cast<const halfx8 *>(lds + ((b ^ (uint32_t)(64 * term)) + (at + (uint32_t)(j * 2048))));
        const uint8_t *q = lds + (b + (b_unit[TB ? 0 : j & (UNITS - 1)] ^ (uint32_t)(64 * term)) +
                                  (at + (uint32_t)(j / UNITS * 256)));
        const shortx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4 *)q);
        const shortx4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4 *)(q + 4 * (W * 16)));
        return __builtin_bit_cast(halfx8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

// `steps` stages from s0, those from `stop` on zeros, by the four wavefronts of
// one of the workgroup's groups; `lds` is the group's.  LOW: the cross products
// have sums of their own, `low`, to which the lower terms' products belong too.  Each
// MFMA rounds its sum four times, and the higher terms' sum is then rounded by a
// third as many.
template <int BM, int BN, int NB, bool TB, bool LOW>
__device__ __forceinline__ void pair_sum(const Operands &p, long long m, uint8_t *lds, int m0, int n0, int s0,
                                         int stop, int steps, floatx4 (&acc)[BM / 32][BN / 32],
                                         floatx4 (&low)[LOW ? BM / 32 : 1][LOW ? BN / 32 : 1])
{
    constexpr int BK = 32, FA = BM / 32, FB = BN / 32;
    constexpr int STAGE = stage_bytes<BM, BN>();
    typedef StageLoads<BM, BN, TB> From;
    constexpr int LOADS = From::LOADS;   // a wavefront's, of a stage
    const uint32_t ring = lds_address(lds);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) & 3);
    From from(p, m, m0, n0, s0, min(p.K, BK * stop), lane, wave);
    const StageLanes<BM, BN, TB> lanes(lane, wave);
    uint32_t to = ring;   // the buffer that the next loads fill
    struct Loads {
        typename From::Stage stage;
        uint32_t to;
    };
    auto loads = [&]() {   // of the next stage
        const Loads L{from.next(), to};
        to = to == ring + (uint32_t)((NB - 1) * STAGE) ? ring : to + STAGE;
        return L;
    };
    auto load = [&](const Loads &L, int i) { from.load(L.stage, L.to, i); };   // load i of the stage

    struct Fragments {
        halfx8 a[2][FA], b[2][FB];
    };
    constexpr int READS = 2 * (FA + FB);
    auto read = [&](uint32_t at, int r, Fragments &f) {   // read r of the stage in the buffer at `at`
        if (r < 2 * FA)
            f.a[r / FA][r % FA] = lanes.read_a(lds, at, r % FA, r / FA);
        else
            f.b[(r - 2 * FA) / FB][(r - 2 * FA) % FB] = lanes.read_b(lds, at, (r - 2 * FA) % FB, (r - 2 * FA) / FB);
    };

#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                asm("v_accvgpr_write_b32 %0, 0" : "=a"(acc[i][j][r]));   // keeps the arrays in the accumulators
                if (LOW)
                    asm("v_accvgpr_write_b32 %0, 0" : "=a"(low[LOW ? i : 0][LOW ? j : 0][r]));
            }

    auto stage = [&](uint32_t next, const Fragments &c, Fragments &n) {
        constexpr int TERMS = LOW ? 4 : 3, MFMAS = TERMS * FA * FB;
        constexpr int FIRST = MFMAS - READS >= LOADS ? READS : 2, EVERY = (MFMAS - FIRST) / LOADS;
        static_assert(EVERY > 0 && READS <= MFMAS, "all issued");
        Loads L;
#pragma unroll
        for (int x = 0; x < MFMAS; ++x) {
            const int i = x / (TERMS * FB), t = x / FB % TERMS, j = x % FB;   // hi hi, lo hi, hi lo, lo lo
            floatx4 &sum = !LOW || t == 0 ? acc[i][j] : low[LOW ? i : 0][LOW ? j : 0];
            sum = OpHalf::mfma(c.a[t & 1][i], c.b[t >> 1][j], sum);
            if (x < READS)
                read(next, x, n);
            if (x == 0)
                L = loads();
            if (x >= FIRST && (x - FIRST) % EVERY == EVERY - 1 && (x - FIRST) / EVERY < LOADS)
                load(L, (x - FIRST) / EVERY);
            // keep this order: the compiler would otherwise cluster the reads and
            // loads, and move MFMAs across the barrier
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    Fragments f0, f1;
#pragma unroll
    for (int st = 0; st < NB; ++st) {
        const Loads L = loads();
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            load(L, i);
    }
    __builtin_amdgcn_s_waitcnt(wait_vmcnt((NB - 1) * LOADS));
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int r = 0; r < READS; ++r)
        read(0, r, f0);
    uint32_t at = 0;   // the buffer of the stage whose fragments are in use
    auto begin = [&]() {
        __builtin_amdgcn_s_waitcnt(wait_vmcnt_lgkm0((NB - 2) * LOADS));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        at = at == (uint32_t)((NB - 1) * STAGE) ? 0u : at + STAGE;
    };
    for (int t = 0; t < steps; t += 2) {
        begin();
        stage(at, f0, f1);
        if (t + 1 < steps) {
            begin();
            stage(at, f1, f0);
        }
    }
    // no load may still be writing LDS, nor a wavefront reading the ring
    __builtin_amdgcn_s_waitcnt(wait_vmcnt_lgkm0(0));
    __builtin_amdgcn_s_barrier();
    dgor_acc_hazard_wait();
}

// The same on a tile of 256 x 256, 128 x 128 a wavefront, whose 32 fragments a stage
// leave no registers for the next stage's: two buffers, and the stage in four
// quadrants of 48 MFMAs, in an order in which a half of the fragments is last
// used long before the next stage wants it.  With A's halves 0 and 1 and B's, f the
// one that the stage begins with and o the other, the quadrants are (0, f), (0, o),
// (1, o), (1, f), and the next stage begins with o.  Meanwhile are read: B's o and
// A's 1 of this stage, then A's 0 and B's o of the next.  Half way through the stage
// nobody reads its buffer any more: the loads of the stage after the next go there in
// the two quadrants that follow, and have the two after that to land.
//
// Why this tile: LDS serves 128 bytes a cycle, of which a stage moves 192 KB here in
// its 3 x 1024 cycles of MFMAs, and 96 KB on 128 x 128 in 768, which is then bound by it.
template <bool TB>
__device__ __forceinline__ void quad_sum(const Operands &p, long long m, uint8_t *lds, int m0, int n0, int s0,
                                         int steps, floatx4 (&acc)[8][8])
{
    constexpr int BK = 32, SIDE = 256, STAGE = stage_bytes<SIDE, SIDE>();
    typedef StageLoads<SIDE, SIDE, TB> From;
    const uint32_t ring = lds_address(lds);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    From from(p, m, m0, n0, s0, min(p.K, BK * (s0 + steps)), lane, wave);
    const StageLanes<SIDE, SIDE, TB> lanes(lane, wave);
    auto load = [&](const typename From::Stage &L, int buffer, int i) {
        from.load(L, ring + (uint32_t)(buffer * STAGE), i);
    };

    // fragments; half h of A's and B's blocks is four
    halfx8 fa[2][8], fb[2][8];
    auto read_a = [&](int buffer, int h, int r) {   // read r of 8 of A's half h
        const int t = r >> 2, i = 4 * h + (r & 3);
        fa[t][i] = lanes.read_a(lds, (uint32_t)(buffer * STAGE), i, t);
    };
    auto read_b = [&](int buffer, int h, int r) {
        const int t = r >> 2, j = 4 * h + (r & 3);
        fb[t][j] = lanes.read_b(lds, (uint32_t)(buffer * STAGE), j, t);
    };

#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                asm("v_accvgpr_write_b32 %0, 0" : "=a"(acc[i][j][r]));   // keeps the array in the accumulators

    // A quadrant: its MFMAs, eight reads between the first of them, and (with
    // loads) the given eight loads between all
    auto quadrant = [&](int ih, int jh, auto reads, auto issue) {
#pragma unroll
        for (int x = 0; x < 48; ++x) {
            const int i = 4 * ih + x / 12, t = x / 4 % 3, j = 4 * jh + x % 4;   // hi hi, lo hi, hi lo
            acc[i][j] = OpHalf::mfma(fa[t == 1][i], fb[t == 2][j], acc[i][j]);
            if (x % 3 == 0 && x / 3 < 8)
                reads(x / 3);
            if (x % 6 == 5)
                issue(x / 6);
            __builtin_amdgcn_sched_barrier(0);   // keep this order
        }
    };
    auto none = [](int) {};
    auto stage = [&](int parity) {   // of the stage: its buffer, and the half of B that it begins with
        const int f = parity, o = 1 - parity;
        quadrant(0, f, [&](int r) { read_b(parity, o, r); }, none);
        quadrant(0, o, [&](int r) { read_a(parity, 1, r); }, none);
        // this stage's reads have returned and the next stage's loads landed,
        // everyone's
        __builtin_amdgcn_s_waitcnt(wait_vmcnt_lgkm0(0));
        __builtin_amdgcn_s_barrier();
        const auto L = from.next();
        __builtin_amdgcn_sched_barrier(0);
        quadrant(1, o, [&](int r) { read_a(o, 0, r); }, [&](int l) { load(L, parity, l); });
        quadrant(1, f, [&](int r) { read_b(o, o, r); }, [&](int l) { load(L, parity, 8 + l); });
    };

#pragma unroll
    for (int st = 0; st < 2; ++st) {
        const auto L = from.next();
#pragma unroll
        for (int i = 0; i < From::LOADS; ++i)
            load(L, st, i);
    }
    __builtin_amdgcn_s_waitcnt(wait_vmcnt(From::LOADS));
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        read_a(0, 0, r);
        read_b(0, 0, r);
    }
    for (int t = 0; t < steps; t += 2) {
        stage(0);
        if (t + 1 < steps)
            stage(1);
    }
    // no load may still be writing LDS, nor a wavefront reading the buffers
    __builtin_amdgcn_s_waitcnt(wait_vmcnt_lgkm0(0));
    __builtin_amdgcn_s_barrier();
    dgor_acc_hazard_wait();
}

// stage_rows of the sum of two sums.
template <int F>
__device__ __forceinline__ void stage_sums(const floatx4 (&acc)[F][F], const floatx4 (&low)[F][F], int round, float *w,
                                           int row, int lane)
{
    const int s16 = lane & 15, g = lane >> 4;
#pragma unroll
    for (int k = 0; k < F / 2; ++k)
        if (round == k) {
#pragma unroll
            for (int ii = 0; ii < 2; ++ii)
#pragma unroll
                for (int j = 0; j < F; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        w[(16 * ii + 4 * g + r) * row + 16 * j + s16] =
                            dgor_acc_read(acc[2 * k + ii][j][r]) + dgor_acc_read(low[2 * k + ii][j][r]);
        }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// GROUPS: groups of four wavefronts, which take halves of a tile's stages on rings
// of their own and add their sums in LDS.  Two on the 64 x 64 tile, whose stages are
// too short for one wavefront a SIMD to cover its own waits.
// LOW: as pair_sum's.
template <int SIDE, int NB, int GROUPS, bool LOW, Which WHICH>
__global__ __launch_bounds__(256 * GROUPS) void newton_schulz_kernel(Operands p, Work work, Finish f)
{
    constexpr bool SYM = WHICH != kUpdate, TB = SYM;
    constexpr int HALF = SIDE / 2, F = HALF / 16;
    constexpr int ROW = HALF + 4, LANES = HALF / 8, STEP = 64 / LANES;
    constexpr int ROWS = 32 / GROUPS;                                // of a round, a group's
    constexpr int BATCH = SIDE == 128 ? 4 : ROWS / STEP < 2 ? 1 : 2;   // rows of a lane at once
    constexpr int RING = NB * stage_bytes<SIDE, SIDE>(), REGION = 32 * ROW;
    static_assert(GROUPS == 1 || F == 2, "a group's sums are one round");
    static_assert(4 * REGION * 4 <= RING && GROUPS * RING <= 160 * 1024, "the epilogue uses the ring's LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[GROUPS * RING];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) & 3);
    const int group = GROUPS == 1 ? 0 : __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 8));
    float *const w = reinterpret_cast<float *>(lds) + wave * REGION;                            // group 0's sums
    float *const own = reinterpret_cast<float *>(lds + group * RING) + wave * REGION;
    // the sum of an element of the wavefront's part of the tile
    auto sum = [&](int at) { return GROUPS == 1 ? w[at] : w[at] + w[RING / 4 + at]; };

    // workgroup ids go round the XCDs: the ones of an XCD take neighbouring tiles
    const int per = work.groups >> 3, rem = work.groups & 7, xcd = (int)blockIdx.x & 7;
    const int me = xcd * per + min(xcd, rem) + ((int)blockIdx.x >> 3);
    const long long all = (long long)(work.tiles - work.whole) * work.stages;
    const long long last = min((long long)(me + 1) * work.run, all);
    long long unit = (long long)me * work.run;
    for (int tile = me;;) {
        int s0 = 0, steps = work.stages;
        long long begin = 0;
        const bool alone = tile < work.whole;
        if (!alone) {
            if (unit >= last)
                break;
            const int t = (int)(unit / work.stages);
            begin = (long long)t * work.stages;
            tile = work.whole + t;
            s0 = (int)(unit - begin);
            steps = (int)min(last - unit, (long long)(work.stages - s0));
            unit += steps;
        }
        const int m = tile / work.per;
        int tm, tn;
        tile_of<SYM>(work, tile - m * work.per, tm, tn);
        floatx4 acc[F][F], low[LOW ? F : 1][LOW ? F : 1];
        if constexpr (SIDE == 256) {
            quad_sum<TB>(p, m, lds, tm * SIDE, tn * SIDE, s0, steps, acc);
        } else {
            const int each = (steps + GROUPS - 1) / GROUPS;
            pair_sum<SIDE, SIDE, NB, TB, LOW>(p, m, lds + group * RING, tm * SIDE, tn * SIDE, s0 + group * each,
                                         min(s0 + steps, s0 + (group + 1) * each), each, acc, low);
        }

        // 32 rows at a time through the wavefront's own part of LDS: a lane has
        // eight columns of every STEP-th row, and then, of what is also written
        // across, eight rows of a column.  A's elements are loaded a batch ahead and
        // before the batch's stores, whose returns they would else wait for (a row
        // at a time a 128 x 128 tile took 12 us more).
        const bool part = steps < work.stages;
        const bool mirrored = SYM && !part && tn < tm, turned = WHICH == kUpdate && !part && f.turned;
        float *slab = work.slabs + (part ? work.slab(me, begin, SIDE * SIDE) : 0);
        const int r0 = ROWS * group + lane / LANES, c = 8 * (lane % LANES);
        const int in = (wave >> 1) * HALF, left = (wave & 1) * HALF;   // in the tile
        const int top = tm * SIDE + in, col = tn * SIDE + left + c;
        const bool polynomial = WHICH == kPolynomial && !part;
        u32x4 with[BATCH][2];
        auto load_with = [&](int first) {   // of the lane's rows from `first` on
#pragma unroll
            for (int q = 0; q < BATCH; ++q) {
                const uint16_t *at = f.with.at(m, min(top + first + r0 + STEP * q, p.M - 1), min(col, p.N - 1) & ~7);
                with[q][0] = *reinterpret_cast<const u32x4 *>(at);
                with[q][1] = *reinterpret_cast<const u32x4 *>(at + 32);
            }
        };
        if (polynomial)
            load_with(0);
#pragma unroll 1
        for (int round = 0; round < F / 2; ++round) {
            if constexpr (LOW)
                stage_sums(acc, low, round, own, ROW, lane);
            else
                stage_rows(acc, round, own, ROW, lane);
            if (GROUPS > 1)
                __syncthreads();
            const int row0 = top + 32 * round;
            if (polynomial) {
#pragma unroll 1
                for (int b = 0; b < ROWS; b += BATCH * STEP) {
                    float v[BATCH][8];
#pragma unroll
                    for (int q = 0; q < BATCH; ++q) {
                        const int r = b + r0 + STEP * q;
                        float a[8], lo[8];
                        unpack8<Half16>(with[q][0], a);
                        unpack8<Half16>(with[q][1], lo);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            a[e] += lo[e];
                            v[q][e] = sum(r * ROW + c + e);
                        }
                        f.value(row0 + r, col, v[q], a);
                        // (rows past the matrix become P's padding, which has to be zeros:
                        // theirs here is b A of its last row, which P's bound does not hold)
                        if (mirrored)
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                w[r * ROW + c + e] = row0 + r < p.M ? v[q][e] : 0.f;
                    }
                    if (GROUPS == 1 && 32 * round + b + BATCH * STEP < HALF)
                        load_with(32 * round + b + BATCH * STEP);
#pragma unroll
                    for (int q = 0; q < BATCH; ++q)
                        if (row0 + b + r0 + STEP * q < p.M && col < p.N)
                            f.store(m, row0 + b + r0 + STEP * q, col, p.N - col, v[q]);
                }
            } else if (!turned) {
#pragma unroll 1
                for (int r = r0; r < ROWS * (group + 1); r += STEP) {
                    if (row0 + r >= p.M || col >= p.N)
                        break;
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = sum(r * ROW + c + e) * (part ? 1.f : f.alpha[0]);
                    if (part)
                        store8_f32(slab + (in + 32 * round + r) * SIDE + left + c, 8, v);
                    else
                        f.store(m, row0 + r, col, p.N - col, v);
                }
            }
            if (mirrored || turned) {   // four lanes a column: 64 bytes of 16-bit results
                if (polynomial) {
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                    if (GROUPS > 1)
                        __syncthreads();   // (both groups' rows)
                }
                const int r = 8 * (lane & 3), row = row0 + r;
#pragma unroll 1
                for (int x = (lane >> 2) + 16 * group; x < HALF; x += 16 * GROUPS) {
                    const int at = tn * SIDE + left + x;
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = polynomial ? w[(r + e) * ROW + x] : f.alpha[0] * sum((r + e) * ROW + x);
                    if (row < p.M && at < p.N)
                        f.store(m, at, row, p.M - row, v);
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        if (alone)
            tile += work.groups;
        // the next tile's loads count in order only after these stores, and fill
        // LDS that other wavefronts may still read
        __builtin_amdgcn_s_waitcnt(wait_vmcnt_lgkm0(0));
        __builtin_amdgcn_s_barrier();
    }
}

// Adds the slabs of the tiles in several runs, in their order: a block of 64 x 64
// a workgroup.
template <int SIDE, bool SYM>
__global__ __launch_bounds__(256) void newton_schulz_join_kernel(Operands p, Work work, Finish f)
{
    constexpr int ACROSS = SIDE / 64, BLOCKS = ACROSS * ACROSS;
    __shared__ float block[64][68];
    const int t = (int)blockIdx.x / BLOCKS, id = (int)blockIdx.x - t * BLOCKS;
    const long long begin = (long long)t * work.stages, end = begin + work.stages;
    const int w0 = (int)(begin / work.run), w1 = (int)((end - 1) / work.run);
    if (w0 == w1)
        return;   // a tile in one run
    const int tile = work.whole + t, m = tile / work.per;
    int tm, tn;
    tile_of<SYM>(work, tile - m * work.per, tm, tn);
    const bool across = f.turned || (SYM && tn < tm);
    const int in = 64 * (id / ACROSS), left = 64 * (id % ACROSS), r0 = tm * SIDE + in, c0 = tn * SIDE + left;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int r = (int)(threadIdx.x >> 3) + 32 * q, c = 8 * (int)(threadIdx.x & 7);
        float v[8] = {};
        if (r0 + r < p.M && c0 + c < p.N) {
            const int at = (in + r) * SIDE + left + c;
            load8_f32(work.slabs + work.slab(w0, begin, SIDE * SIDE) + at, 8, v);
            for (int s = w0 + 1; s <= w1; ++s) {
                float u[8];
                load8_f32(work.slabs + work.slab(s, begin, SIDE * SIDE) + at, 8, u);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] += u[e];
            }
        }
        const bool inside = r0 + r < p.M && c0 + c < p.N;
        float a[8] = {};
        if (f.polynomial && inside)
            f.with.load8(m, r0 + r, c0 + c, a);
        f.value(r0 + r, c0 + c, v, a);
        if (across)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                block[r][c + e] = v[e];
        if (!f.turned && inside)
            f.store(m, r0 + r, c0 + c, p.N - c0 - c, v);
    }
    if (!across)
        return;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int c = (int)(threadIdx.x >> 3) + 32 * q, r = 8 * (int)(threadIdx.x & 7);
        if (r0 + r < p.M && c0 + c < p.N) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = block[r + e][c];
            f.store(m, c0 + c, r0 + r, p.M - r0 - r, v);
        }
    }
}

// --------------------------------------------------------- small matrices --
//
// A matrix that fits LDS in two terms next to its A: all steps in one launch, a
// workgroup of 16 wavefronts a matrix.  Bound by the latency of a product's chain,
// LDS to MFMA to LDS and a barrier, where the launches of the kernels above, three a
// step, take 5 us each (five steps of 64 x 64: 29 us, and 76).  A lane's results are
// four neighbours of the transpose, so A and P, symmetric, are written four at a time
// and X with its columns as the first operand.
//
// X is planes of 32 columns, A and P after it likewise: row r of a plane 128 bytes,
// higher terms and then lower ones, unit c at 8 r + (c ^ ((r >> 1) & 7)).  Rows and
// columns up to multiples of 32 are zeros.
struct SmallStep {
    float gram, alpha[2], beta[2], diagonal[2], next;   // Finish's; of A's, P's and the next X's sums
};
// T: planes of 32 T rows, 0 where that is known to the call alone.
template <int T>
struct Planes {
    uint8_t *lds;
    int bytes, s16, g;        // of a plane; the lane's row or column, and its group
    uint32_t rows, cols[2];   // the lane's part of its fragments' addresses,
    uint32_t four, one[2];    // and of its results'
    __device__ __forceinline__ Planes(uint8_t *at, int size, int lane)
        : lds(at), bytes(size), s16(lane & 15), g(lane >> 4)
    {
        rows = (uint32_t)(s16 * 128 + ((g ^ ((s16 >> 1) & 7)) * 16));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = 8 * g + 4 * h + (s16 >> 2);
            cols[h] = (uint32_t)(k * 128 + ((((s16 & 3) >> 1) ^ ((k >> 1) & 7)) * 16) + 8 * (s16 & 1));
            one[h] = (uint32_t)((4 * g + 2 * h) * 128 + (((s16 >> 3) ^ ((2 * g + h) & 7)) * 16) + 2 * (s16 & 7));
        }
        four = (uint32_t)(s16 * 128 + (((g >> 1) ^ ((s16 >> 1) & 7)) * 16) + 8 * (g & 1));
    }
    __device__ __forceinline__ int plane() const { return T ? 4096 * T : bytes; }
    // element (r, c) of planes at `base`; its lower term is 64 bytes on, by an XOR
    __device__ __forceinline__ uint8_t *place(uint8_t *base, int r, int c) const
    {
        return base + (c >> 5) * plane() + r * 128 + ((((c & 31) >> 3) ^ ((r >> 1) & 7)) * 16) + 2 * (c & 7);
    }
    __device__ __forceinline__ uint8_t *lower(const uint8_t *q) const { return lds + ((uint32_t)(q - lds) ^ 64u); }
    __device__ __forceinline__ void put(uint8_t *base, int r, int c, float y) const
    {
        uint8_t *q = place(base, r, c);
        const _Float16 hi = (_Float16)y;
        *reinterpret_cast<_Float16 *>(q) = hi;
        *reinterpret_cast<_Float16 *>(lower(q)) = (_Float16)(y - (float)hi);
    }
    // The 16 x 16 block (bi, bj) of planes at base from its transpose as the matrix
    // cores give it: the lane's row 16 bi + s16, four neighbours from 16 bj + 4 g.
    __device__ __forceinline__ uint8_t *place4(uint8_t *base, int bi, int bj, int term) const
    {
        return base + ((bj >> 1) * plane() + 2048 * bi) + (four ^ (32u * (bj & 1) ^ 64u * term));
    }
    __device__ __forceinline__ void put4(uint8_t *base, int bi, int bj, floatx4 y) const
    {
        halfx4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = (_Float16)y[e];
            lo[e] = (_Float16)(y[e] - (float)hi[e]);
        }
        *reinterpret_cast<halfx4 *>(place4(base, bi, bj, 0)) = hi;
        *reinterpret_cast<halfx4 *>(place4(base, bi, bj, 1)) = lo;
    }
    __device__ __forceinline__ floatx4 get4(uint8_t *base, int bi, int bj) const
    {
        const halfx4 hi = *reinterpret_cast<const halfx4 *>(place4(base, bi, bj, 0));
        const halfx4 lo = *reinterpret_cast<const halfx4 *>(place4(base, bi, bj, 1));
        floatx4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = (float)hi[e] + (float)lo[e];
        return y;
    }
    // as it is: the lane's column 16 bj + s16, rows from 16 bi + 4 g
    __device__ __forceinline__ void put_turned(uint8_t *base, int bi, int bj, floatx4 y) const
    {
        uint8_t *q = base + ((bj >> 1) * plane() + 2048 * bi);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t at = one[e >> 1] ^ 32u * (bj & 1);
            const _Float16 hi = (_Float16)y[e];
            *reinterpret_cast<_Float16 *>(q + at + 128 * (e & 1)) = hi;
            *reinterpret_cast<_Float16 *>(q + (at ^ 64u) + 128 * (e & 1)) = (_Float16)(y[e] - (float)hi);
        }
    }
    // four neighbouring elements of P, of the sums v of A A and A's own
    // (of block (bi, bj), as it is or its transpose: both are symmetric)
    __device__ __forceinline__ floatx4 polynomial(const SmallStep &k, bool diagonal, floatx4 v, floatx4 a) const
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool on = diagonal && s16 == 4 * g + e;
            const float rest = __builtin_fmaf(k.alpha[1], v[e], __builtin_fmaf(k.beta[1], a[e], on ? k.diagonal[1] : 0.f));
            v[e] = __builtin_fmaf(k.alpha[0], v[e], __builtin_fmaf(k.beta[0], a[e], on ? k.diagonal[0] : 0.f)) + rest;
        }
        return v;
    }
    // Fragments: rows 16 b .. of planes at base, k 32 t ..; and columns 16 b ...  A
    // lane's part of the address is found once: planes start on 128 bytes, so what the
    // term and b change in it are XORs, and the rest is the same in all lanes.
    __device__ __forceinline__ halfx8 along(const uint8_t *base, int b, int t, int term) const
    {
        return *reinterpret_cast<const halfx8 *>(base + (t * plane() + 2048 * b) + (rows ^ (64u * term)));
    }
    __device__ __forceinline__ halfx8 across(const uint8_t *base, int b, int t, int term) const
    {
        const uint8_t *q = base + ((b >> 1) * plane() + 4096 * t);
        const uint32_t flip = 64u * term ^ 32u * (b & 1);
        shortx4 part[2];
        part[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4 *)(q + (cols[0] ^ flip)));
        part[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4 *)(q + (cols[1] ^ flip)));
        return __builtin_bit_cast(halfx8, __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
    // the sum over `stages` of a block: all four products, the cross ones apart, and
    // two halves of the others, for fewer roundings of each (KNOWN: T stages)
    template <bool KNOWN = false, class A, class B>
    static __device__ __forceinline__ floatx4 block(int stages, A a_of, B b_of)
    {
        floatx4 sum = {0.f, 0.f, 0.f, 0.f}, other = sum, low = sum;
        auto add = [&](int t, floatx4 &to) {
            const halfx8 a0 = a_of(t, 0), b0 = b_of(t, 0), a1 = a_of(t, 1), b1 = b_of(t, 1);
            to = OpHalf::mfma(a0, b0, to);
            low = OpHalf::mfma(a1, b1, low);   // (counts in sums of few products)
            low = OpHalf::mfma(a1, b0, low);
            low = OpHalf::mfma(a0, b1, low);
        };
        auto both = [&](int t, int half) {
            add(t, sum);
            if (half + t < stages)
                add(half + t, other);
        };
        if constexpr (T != 0 && KNOWN) {
#pragma unroll
            for (int t = 0; t < (T + 1) / 2; ++t)
                both(t, (T + 1) / 2);
        } else {
            const int half = (stages + 1) / 2;
            for (int t = 0; t < half; ++t)
                both(t, half);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
            sum[r] = sum[r] + other[r] + low[r];
        return sum;
    }
};

struct Small {
    Source g;
    int m, n, mp, np;   // mp, np: padded to multiples of 32
    bool turned_in, turned_out;
    double eps, by;
    int steps;
    void *out;
    int out_ld, fmt;
    long long out_matrix;
    SmallStep step[GEMM_MAX_STEPS];
};

__global__ __launch_bounds__(64 * kSmallWaves) void newton_schulz_small_kernel(Small p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kSmallBytes];
    __shared__ double sums[kSmallWaves];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const long long matrix = blockIdx.x;
    const int mp = p.mp, plane = mp * 128, nb = (p.n + 15) / 16;
    int mb = (p.m + 15) / 16;
    uint8_t *const xs = lds, *const as = lds + p.np / 32 * plane;
    Planes<0> w(lds, plane, lane);

    // G, its norm, X
    for (int i = threadIdx.x; i < (p.np + mp) / 32 * plane / 16; i += 64 * kSmallWaves)
        *reinterpret_cast<u32x4 *>(lds + 16 * i) = u32x4{0u, 0u, 0u, 0u};
    const int across = (p.g.cols + 7) / 8, units = across * p.g.rows;
    float f[kSmallUnits][8];
    double v = 0;
#pragma unroll
    for (int t = 0; t < kSmallUnits; ++t) {
        const int id = (int)threadIdx.x + 64 * kSmallWaves * t;
        if (id < units) {
            p.g.load8(matrix, id / across, 8 * (id % across), f[t]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v += (double)f[t][e] * (double)f[t][e];
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v += __shfl_xor(v, o, 64);
    if (lane == 0)
        sums[wave] = v;
    __syncthreads();   // and LDS is zero
    v = sums[0];
#pragma unroll
    for (int i = 1; i < kSmallWaves; ++i)
        v += sums[i];
    const double factor = factor_of(p.by, v, p.eps);
#pragma unroll
    for (int t = 0; t < kSmallUnits; ++t) {
        const int id = (int)threadIdx.x + 64 * kSmallWaves * t;
        if (id < units) {
            const int r = id / across, c = 8 * (id % across);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < p.g.cols)
                    w.put(xs, p.turned_in ? c + e : r, p.turned_in ? r : c + e, (float)(f[t][e] * factor));
        }
    }
    __syncthreads();

    constexpr int SQUARES = 4;   // blocks of A a wavefront computes, of mp = 128
#pragma unroll 1
    for (int i = 0; i < p.steps; ++i) {
        // (else every block's addresses are found once, kept, and spilled)
        asm volatile("" : "+v"(w.s16), "+v"(w.g), "+v"(w.rows), "+v"(w.cols[0]), "+v"(w.cols[1]), "+v"(w.four), "+s"(mb));
        const int squares = mb * mb;
        // read where the argument lies: an index into it that is not a constant
        // puts a copy of it into scratch memory
        typedef const __attribute__((address_space(4))) char ArgumentByte;
        typedef const __attribute__((address_space(4))) float ArgumentFloat;
        ArgumentFloat *at = (ArgumentFloat *)((ArgumentByte *)__builtin_amdgcn_kernarg_segment_ptr() +
                                              offsetof(Small, step) + i * sizeof(SmallStep));
        static_assert(sizeof(SmallStep) == 8 * sizeof(float), "");
        const SmallStep k = {at[0], {at[1], at[2]}, {at[3], at[4]}, {at[5], at[6]}, at[7]};
        for (int id = wave; id < squares; id += kSmallWaves) {
            const int bi = id / mb, bj = id % mb;
            const floatx4 v4 = Planes<0>::block(p.np / 32, [&](int t, int term) { return w.along(xs, bi, t, term); },
                                     [&](int t, int term) { return w.along(xs, bj, t, term); });
            w.put4(as, bj, bi, k.gram * v4);   // (symmetric)
        }
        __syncthreads();
        floatx4 held[kSmallBlocks];
#pragma unroll
        for (int b = 0; b < SQUARES; ++b) {
            const int id = wave + kSmallWaves * b, bi = id / mb, bj = id % mb;
            if (id < squares) {
                held[b] = Planes<0>::block(mp / 32, [&](int t, int term) { return w.along(as, bi, t, term); },
                                [&](int t, int term) { return w.along(as, bj, t, term); });
                held[b] = w.polynomial(k, bi == bj, held[b], w.get4(as, bj, bi));
            }
        }
        __syncthreads();   // A has been read
#pragma unroll
        for (int b = 0; b < SQUARES; ++b) {
            const int id = wave + kSmallWaves * b, bi = id / mb, bj = id % mb;
            if (id < squares)
                w.put4(as, bj, bi, held[b]);
        }
        __syncthreads();
#pragma unroll
        for (int b = 0; b < kSmallBlocks; ++b) {
            const int id = wave + kSmallWaves * b, bi = id % mb, bj = id / mb;
            if (id < mb * nb) {
                // (X's columns first: a lane's four are neighbours)
                held[b] = Planes<0>::block(mp / 32, [&](int t, int term) { return w.across(xs, bj, t, term); },
                                        [&](int t, int term) { return w.along(as, bi, t, term); });
            }
        }
        __syncthreads();   // X has been read
#pragma unroll
        for (int b = 0; b < kSmallBlocks; ++b) {
            const int id = wave + kSmallWaves * b, bi = id % mb, bj = id / mb;
            if (id < mb * nb) {
                const int row = 16 * bi + w.s16, col = 16 * bj + 4 * w.g;
                const floatx4 y = k.next * held[b];
                if (i + 1 < p.steps)
                    w.put4(xs, bi, bj, y);
                else   // the result, as it is stored
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (row < p.m && col + e < p.n)
                            reinterpret_cast<float *>(xs)[p.turned_out ? (col + e) * p.m + row : row * p.n + col + e] = y[e];
            }
        }
        __syncthreads();
    }
    const int cols = p.turned_out ? p.m : p.n, rows = p.turned_out ? p.n : p.m, wide = (cols + 7) / 8;
    for (int id = threadIdx.x; id < wide * rows; id += 64 * kSmallWaves) {
        const int r = id / wide, c = 8 * (id % wide);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            y[e] = reinterpret_cast<const float *>(xs)[r * cols + min(c + e, cols - 1)];
        store8_of(p.fmt, p.out, matrix * p.out_matrix + (size_t)r * p.out_ld + c, cols - c, y);
    }
}

// ----------------------------------------------------- matrices of few rows --
//
// Up to 128 rows, in more columns than one workgroup is best for: X stays in strips
// of columns, a workgroup each, and a step is one launch.  It adds the strips' parts
// of A = X X^T, computes P (each strip's workgroup all of it), its strip of P X, and
// that strip's part of the next A.  Planes are as above; a strip lies in the
// workspace as LDS holds it, a part of A as the lanes hold the blocks on and below
// the diagonal.  T is m's 32-row blocks: with it in the code the sums' reads have
// constant offsets and are all in flight at once (a step 13 us, 15.5 without).
// Bound by latency as well: of 13 us a step (8 of 128 x 256; three launches took 18)
// 3 go into the parts of A, 2 into placing A, 2.4 each into the two products, 1.4 and
// 1 into placing P and X, 1.5 into what is left for the next step.
struct Strips {
    int m, n, width, strips;       // width: a strip's columns, a multiple of 32
    bool turned;                   // in: X is G's transpose; out: the result's
    uint8_t *images;               // X's strips
    float *parts;                  // of the next A
};

__device__ __forceinline__ void block_of(int id, int &bi, int &bj)   // on and below the diagonal
{
    for (bi = 0; id > bi; id -= ++bi)
        ;
    bj = id;
}

// A strip of X and its part of A, from LDS to the workspace.
template <int T>
__device__ __forceinline__ void leave_strip(const Strips &p, const Planes<T> &w, const uint8_t *xs, int wave)
{
    const int lane = threadIdx.x & 63, mb = (p.m + 15) / 16, lower = mb * (mb + 1) / 2, bytes = 128 * T * p.width;
    uint8_t *const image = p.images + (size_t)blockIdx.x * bytes;
    for (int i = 16 * threadIdx.x; i < bytes; i += 16 * 64 * kSmallWaves)
        *reinterpret_cast<u32x4 *>(image + i) = *reinterpret_cast<const u32x4 *>(xs + i);
    float *const part = p.parts + (size_t)blockIdx.x * lower * 256;
    for (int id = wave; id < lower; id += kSmallWaves) {
        int bi, bj;
        block_of(id, bi, bj);
        *reinterpret_cast<floatx4 *>(part + 256 * id + 4 * lane) =
            Planes<T>::block(p.width / 32, [&](int t, int term) { return w.along(xs, bi, t, term); },
                          [&](int t, int term) { return w.along(xs, bj, t, term); });
    }
}

template <int T>
__global__ __launch_bounds__(64 * kSmallWaves) void strips_start_kernel(Strips p, Source g, double eps, double by)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kSmallBytes];
    __shared__ double sums[kSmallWaves];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const long long matrix = blockIdx.x / p.strips;
    const int first = (int)(blockIdx.x - matrix * p.strips) * p.width, plane = 4096 * T;
    const Planes<T> w(lds, plane, lane);
    for (int i = 16 * threadIdx.x; i < p.width / 32 * plane; i += 16 * 64 * kSmallWaves)
        *reinterpret_cast<u32x4 *>(lds + i) = u32x4{0u, 0u, 0u, 0u};
    // the norm, of the whole matrix: in every strip's workgroup the same
    double v = 0;
    const int across = (g.cols + 7) / 8, units = across * g.rows;
    const auto add = [&](auto fmt, auto whole) {   // four units' loads in flight at once
        constexpr int AT_ONCE = 4;
        for (int id0 = threadIdx.x; id0 < units; id0 += 64 * kSmallWaves * AT_ONCE) {
            float f[AT_ONCE][8];
#pragma unroll
            for (int t = 0; t < AT_ONCE; ++t) {
                const int id = min(id0 + 64 * kSmallWaves * t, units - 1), r = id / across, c = 8 * (id - r * across);
                load8_of(fmt, g.p, matrix * g.matrix + (size_t)r * g.ld + c, whole ? 8 : g.cols - c, f[t]);
            }
#pragma unroll
            for (int t = 0; t < AT_ONCE; ++t)
                if (id0 + 64 * kSmallWaves * t < units)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v += (double)f[t][e] * (double)f[t][e];
        }
    };
    const auto add_of = [&](auto fmt) {
        if (g.cols % 8 == 0)
            add(fmt, std::true_type());
        else
            add(fmt, std::false_type());
    };
    switch (g.fmt) {
    case kF32: add_of(std::integral_constant<int, kF32>()); break;
    case kF16: add_of(std::integral_constant<int, kF16>()); break;
    default: add_of(std::integral_constant<int, kBF16>()); break;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v += __shfl_xor(v, o, 64);
    if (lane == 0)
        sums[wave] = v;
    __syncthreads();   // and LDS is zero
    v = sums[0];
#pragma unroll
    for (int i = 1; i < kSmallWaves; ++i)
        v += sums[i];
    const double factor = factor_of(by, v, eps);
    // the strip's rows and units of G: `first` of them left out
    const int r0 = p.turned ? first : 0, c0 = p.turned ? 0 : first;
    const int rows = p.turned ? min(p.width, g.rows - r0) : g.rows, cols = p.turned ? g.cols : min(p.width, g.cols - c0);
    const int wide = (cols + 7) / 8;
    for (int id = threadIdx.x; id < wide * rows; id += 64 * kSmallWaves) {
        const int r = id / wide, c = 8 * (id % wide);
        float f[8];
        g.load8(matrix, r0 + r, c0 + c, f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < cols)
                w.put(lds, p.turned ? c + e : r, p.turned ? r : c + e, (float)(f[e] * factor));
    }
    __syncthreads();
    leave_strip(p, w, lds, wave);
}

struct Result {
    void *p;
    int ld, fmt;
    long long matrix;
};

template <int T, bool LAST>
__global__ __launch_bounds__(64 * kSmallWaves) void strips_step_kernel(Strips p, const float *parts, SmallStep k, Result out)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kSmallBytes];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const long long matrix = blockIdx.x / p.strips;
    const int strip = (int)(blockIdx.x - matrix * p.strips), plane = 4096 * T;
    const int mb = (p.m + 15) / 16, lower = mb * (mb + 1) / 2, bytes = p.width / 32 * plane;
    uint8_t *const xs = lds, *const as = lds + bytes;
    const Planes<T> w(lds, plane, lane);
    for (int i = 16 * threadIdx.x; i < T * plane; i += 16 * 64 * kSmallWaves)
        *reinterpret_cast<u32x4 *>(as + i) = u32x4{0u, 0u, 0u, 0u};
    constexpr int SQUARES = (T * (2 * T + 1) + kSmallWaves - 1) / kSmallWaves;   // blocks on and below the diagonal a wavefront holds
    floatx4 held[kSmallBlocks];
    parts += (size_t)matrix * p.strips * lower * 256 + 4 * lane;
    // all loads of four strips in flight at once: those past the last strip are the
    // last one's, and not added
#pragma unroll
    for (int b = 0; b < SQUARES; ++b)
        held[b] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < p.strips; s0 += 4) {
        floatx4 v[SQUARES][4];
#pragma unroll
        for (int b = 0; b < SQUARES; ++b)
            if (wave + kSmallWaves * b < lower)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    v[b][s] = *reinterpret_cast<const floatx4 *>(
                        parts + ((size_t)min(s0 + s, p.strips - 1) * lower + wave + kSmallWaves * b) * 256);
#pragma unroll
        for (int b = 0; b < SQUARES; ++b)
            if (wave + kSmallWaves * b < lower)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    held[b] += s0 + s < p.strips ? v[b][s] : floatx4{0.f, 0.f, 0.f, 0.f};
    }
    __syncthreads();   // A's planes are zero
    // a symmetric matrix's blocks, to both places
    auto put_squares = [&](float by) {
#pragma unroll
        for (int b = 0; b < SQUARES; ++b) {
            const int id = wave + kSmallWaves * b;
            if (id < lower) {
                int bi, bj;
                block_of(id, bi, bj);
                w.put4(as, bj, bi, by * held[b]);
                if (bi != bj)
                    w.put_turned(as, bi, bj, by * held[b]);
            }
        }
    };
    put_squares(k.gram);
    // X is on its way while P is computed
    u32x4 strip_x[kStripUnits];
    const uint8_t *const image = p.images + (size_t)blockIdx.x * bytes;
#pragma unroll
    for (int i = 0; i < kStripUnits; ++i) {
        const int at = 16 * ((int)threadIdx.x + 64 * kSmallWaves * i);
        if (at < bytes)
            strip_x[i] = *reinterpret_cast<const u32x4 *>(image + at);
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < SQUARES; ++b) {
        const int id = wave + kSmallWaves * b;
        if (id < lower) {
            int bi, bj;
            block_of(id, bi, bj);
            held[b] = Planes<T>::template block<true>(T, [&](int t, int term) { return w.along(as, bi, t, term); },
                                    [&](int t, int term) { return w.along(as, bj, t, term); });
            held[b] = w.polynomial(k, bi == bj, held[b], w.get4(as, bj, bi));
        }
    }
#pragma unroll
    for (int i = 0; i < kStripUnits; ++i) {
        const int at = 16 * ((int)threadIdx.x + 64 * kSmallWaves * i);
        if (at < bytes)
            *reinterpret_cast<u32x4 *>(xs + at) = strip_x[i];
    }
    __syncthreads();   // A has been read
    put_squares(1.f);
    __syncthreads();
    const int blocks = mb * (p.width / 16);
#pragma unroll
    for (int b = 0; b < kSmallBlocks; ++b) {
        const int id = wave + kSmallWaves * b, bi = id % mb, bj = id / mb;
        if (id < blocks)
            held[b] = Planes<T>::template block<true>(T, [&](int t, int term) { return w.across(xs, bj, t, term); },
                                    [&](int t, int term) { return w.along(as, bi, t, term); });
    }
    __syncthreads();   // X has been read
    const int first = strip * p.width, inside = min(p.width, p.n - first);
#pragma unroll
    for (int b = 0; b < kSmallBlocks; ++b) {
        const int id = wave + kSmallWaves * b, bi = id % mb, bj = id / mb;
        if (id < blocks) {
            const int row = 16 * bi + w.s16, col = 16 * bj + 4 * w.g;
            const floatx4 y = k.next * held[b];
            if (!LAST)
                w.put4(xs, bi, bj, y);
            else   // the result, as it is stored
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (row < p.m && col + e < inside)
                        reinterpret_cast<float *>(xs)[p.turned ? (col + e) * p.m + row : row * inside + col + e] = y[e];
        }
    }
    __syncthreads();
    if (!LAST) {
        leave_strip(p, w, xs, wave);
        return;
    }
    const int cols = p.turned ? p.m : inside, rows = p.turned ? inside : p.m, wide = (cols + 7) / 8;
    const size_t at = matrix * out.matrix + (p.turned ? (size_t)first * out.ld : (size_t)first);
    for (int id = threadIdx.x; id < wide * rows; id += 64 * kSmallWaves) {
        const int r = id / wide, c = 8 * (id % wide);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            y[e] = reinterpret_cast<const float *>(xs)[r * cols + min(c + e, cols - 1)];
        store8_of(out.fmt, out.p, at + (size_t)r * out.ld + c, cols - c, y);
    }
}

// ------------------------------------------------------------------- host --

template <int SIDE, int NB, int GROUPS, bool LOW = false>
hipError_t launch_as(Which which, const Operands &p, const Work &w, bool joined, const Finish &f, hipStream_t s)
{
    const dim3 grid((unsigned)w.groups), blocks((unsigned)((w.tiles - w.whole) * (SIDE / 64) * (SIDE / 64)));
    const dim3 threads(256 * GROUPS);
    if (which == kUpdate)
        hipLaunchKernelGGL((newton_schulz_kernel<SIDE, NB, GROUPS, LOW, kUpdate>), grid, threads, 0, s, p, w, f);
    else if (which == kPolynomial)
        hipLaunchKernelGGL((newton_schulz_kernel<SIDE, NB, GROUPS, LOW, kPolynomial>), grid, threads, 0, s, p, w, f);
    else
        hipLaunchKernelGGL((newton_schulz_kernel<SIDE, NB, GROUPS, LOW, kGram>), grid, threads, 0, s, p, w, f);
    if (joined && which == kUpdate)
        hipLaunchKernelGGL((newton_schulz_join_kernel<SIDE, false>), blocks, dim3(256), 0, s, p, w, f);
    else if (joined)
        hipLaunchKernelGGL((newton_schulz_join_kernel<SIDE, true>), blocks, dim3(256), 0, s, p, w, f);
    return hipGetLastError();
}

// Up to this many rows the sums are short enough for their few products' rounding to
// show: 20 x 1587 errs by 1.5e-6, and with LOW, at 10% of the time, by 1.0e-6 (FP32
// products: 1.0e-6).  Past it FP32's own sums err more (777 x 1033: 2.8e-6 and 1.7e-6
// without).
constexpr int kFewRows = 128;

hipError_t launch(Which which, const Pair &a, const Pair &b, int m, int n, int batch, const Way &way, float *slabs,
                  const Finish &f, hipStream_t s)
{
    Operands p{m, results_cols(which, m, n), which == kGram ? n : m, a, b};
    Work w;
    w.per = (int)tiles_of(which, m, n, way.tile);
    w.tiles = batch * w.per;
    w.stages = ceil_div(p.K, 32);
    w.tiles_m = ceil_div(p.M, side_of(way.tile)), w.tiles_n = ceil_div(p.N, side_of(way.tile));
    w.groups = way.groups, w.whole = way.whole, w.run = way.run;
    w.slabs = slabs;
    switch (way.tile) {
    case kTile256: return launch_as<256, 2, 1>(which, p, w, way.joined, f, s);
    case kTile128: return launch_as<128, 4, 1>(which, p, w, way.joined, f, s);
    case kTile64:
        return m <= kFewRows ? launch_as<64, 4, 2, true>(which, p, w, way.joined, f, s)
                             : launch_as<64, 4, 2>(which, p, w, way.joined, f, s);
    }
    return hipErrorInvalidValue;
}

int run(int fmt, const gemm_orthogonalize_params *q, const void *G, void *O, void *ws, size_t ws_bytes, void *stream)
{
    Layout l;
    const int rc = lay_out(q, l);
    if (rc != GEMM_OK)
        return rc;
    if (results_overlap(*q))
        return GEMM_ERR_INVALID_LAYOUT;
    if (q->batch == 0 || q->M == 0 || q->N == 0)
        return GEMM_OK;
    if (!G || !O)
        return GEMM_ERR_NULL_PTR;
    if (l.bytes && (!ws || ws_bytes < l.bytes || ((uintptr_t)ws & (kWsAlign - 1)) != 0))
        return GEMM_ERR_WORKSPACE;
    const int dev = device_status();
    if (dev != GEMM_OK)
        return dev;
    hipStream_t s = (hipStream_t)stream;
    uint8_t *base = (uint8_t *)ws;
    const int batch = q->batch;
    const auto hold = [](float (&to)[2], double v) {
        to[0] = (float)v;
        to[1] = (float)(v - to[0]);
    };
    // what the sums of step i's products are multiplied by
    const auto gram_of = [&](int i) { return (float)std::ldexp(1.0, l.step[i].gram - 2 * l.step[i].x); };
    const auto next_of = [&](int i) {
        const int from = l.step[i].poly + l.step[i].x;
        return (float)(i + 1 < q->steps ? std::ldexp(1.0, l.step[i + 1].x - from) : l.last);
    };
    const auto polynomial_of = [&](int i, auto &f) {
        const Step &k = l.step[i];
        hold(f.alpha, std::ldexp(k.c, k.poly - 2 * k.gram));
        hold(f.beta, std::ldexp(k.b, k.poly - k.gram));
        hold(f.diagonal, std::ldexp(k.a, k.poly));
    };
    const bool t = q->op_g == GEMM_OP_T;
    const Source g{G, t ? q->N : q->M, t ? q->M : q->N, q->ldg, batch > 1 ? q->stride_g : 0, fmt};
    if (l.small) {
        Small p{};
        p.g = g;
        p.m = l.m, p.n = l.n, p.mp = (l.m + 31) / 32 * 32, p.np = (l.n + 31) / 32 * 32;
        p.turned_in = l.turned_in, p.turned_out = l.turned_out;
        p.eps = q->eps, p.by = std::ldexp(1.0, l.step[0].x);
        p.steps = q->steps;
        p.out = O, p.out_ld = q->ldo, p.out_matrix = batch > 1 ? q->stride_o : 0, p.fmt = fmt;
        for (int i = 0; i < q->steps; ++i) {
            polynomial_of(i, p.step[i]);
            p.step[i].gram = gram_of(i), p.step[i].next = next_of(i);
        }
        hipLaunchKernelGGL(newton_schulz_small_kernel, dim3((unsigned)batch), dim3(64 * kSmallWaves), 0, s, p);
        return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
    }
    if (l.strips) {
        Strips p{l.m, l.n, l.width, l.strips, l.turned_in, base + l.x[0], nullptr};
        float *const parts[2] = {(float *)(base + l.gram), (float *)(base + l.poly)};
        const Result out{O, q->ldo, fmt, batch > 1 ? q->stride_o : 0};
        const auto steps = [&](auto planes) {
            constexpr int T = decltype(planes)::value;
            const dim3 groups((unsigned)(batch * l.strips)), threads(64 * kSmallWaves);
            p.parts = parts[0];
            hipLaunchKernelGGL(strips_start_kernel<T>, groups, threads, 0, s, p, g, q->eps, std::ldexp(1.0, l.step[0].x));
            p.turned = l.turned_out;
            for (int i = 0; i < q->steps; ++i) {
                SmallStep k;
                polynomial_of(i, k);
                k.gram = gram_of(i), k.next = next_of(i);
                p.parts = parts[(i + 1) & 1];
                const float *from = parts[i & 1];
                if (i + 1 < q->steps)
                    hipLaunchKernelGGL((strips_step_kernel<T, false>), groups, threads, 0, s, p, from, k, out);
                else
                    hipLaunchKernelGGL((strips_step_kernel<T, true>), groups, threads, 0, s, p, from, k, out);
            }
        };
        switch (l.mp / 32) {
        case 1: steps(std::integral_constant<int, 1>()); break;
        case 2: steps(std::integral_constant<int, 2>()); break;
        case 3: steps(std::integral_constant<int, 3>()); break;
        default: steps(std::integral_constant<int, 4>()); break;
        }
        return hipGetLastError() == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
    }
    const auto pair = [&](size_t at, int ld) {
        return Pair{(uint16_t *)(base + at), (long long)l.m * ld, ld};
    };
    const Pair x[2] = {pair(l.x[0], l.ldx), pair(l.x[1], l.ldx)}, gram = pair(l.gram, l.lda), poly = pair(l.poly, l.lda);

    double *sums = (double *)(base + l.sums);
    hipLaunchKernelGGL(squares_kernel, dim3((unsigned)(batch * l.blocks)), dim3(256), 0, s, g, l.blocks, l.lg, sums);
    const int across = ceil_div(g.cols, 64), per = across * ceil_div(g.rows, 64);
    hipLaunchKernelGGL(start_kernel, dim3((unsigned)(batch * per)), dim3(256), 0, s, g, x[0], sums, l.blocks, q->eps,
                       std::ldexp(1.0, l.step[0].x), across, per, l.turned_in);
    hipError_t err = hipGetLastError();

    const auto product = [&](Which which, const Pair &a, const Pair &b, const Finish &f) {
        return launch(which, a, b, l.m, l.n, batch, l.way[which], (float *)(base + l.part), f, s);
    };
    for (int i = 0; i < q->steps && err == hipSuccess; ++i) {
        const Pair &now = x[i & 1], &next = x[(i + 1) & 1];
        Finish f{};
        f.alpha[0] = gram_of(i);
        f.to = gram;
        err = product(kGram, now, now, f);
        if (err != hipSuccess)
            break;
        f.polynomial = true;
        polynomial_of(i, f);
        f.with = gram, f.to = poly;
        err = product(kPolynomial, gram, gram, f);
        if (err != hipSuccess)
            break;
        f = Finish{};
        f.alpha[0] = next_of(i);
        f.to = next;
        if (i + 1 == q->steps) {
            f.out = O, f.out_ld = q->ldo, f.out_matrix = batch > 1 ? q->stride_o : 0;
            f.fmt = fmt, f.turned = l.turned_out;
        }
        err = product(kUpdate, poly, now, f);
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
    dgor::newton_schulz::Layout l;
    const int rc = dgor::newton_schulz::lay_out(params, l);
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
