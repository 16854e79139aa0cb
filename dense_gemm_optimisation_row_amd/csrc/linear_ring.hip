// The dense-layer products of 16-byte aligned operands: tiles of 256 x 256,
// 256 x 128, 128 x 128, 128 x 64 and 64 x 64, loaded straight from global memory into
// LDS rings 32 k deep, FP32 sums on v_mfma_f32_16x16x32, and the epilogue of
// epilogue.h on whole rows.
//
// Four wavefronts, each a quarter of the tile in 16 x 16 blocks: 8 x 8 of them
// (all 256 accumulator registers, one workgroup a compute unit), 8 x 4 (one),
// 4 x 4, 4 x 2 or 2 x 2 (two, which cover each other's waits).
// Loads: one instruction moves 64 lanes x 16 bytes into 1 KB of LDS, lane p
// at byte 16 p; the layout is chosen by permuting the sources, and a lane
// whose offset is out of range writes zeros, which fills every edge.
//
// A stage of an operand whose rows run along the outputs (B as K x N, A as
// K x M) is kept as two halves of the tile's columns, each 32 k rows of W units
// of 16 bytes, unit u of row k at W k + (u ^ x(k)), x(k) = 2 (k & 3) + 8 ((k >> 3) & 1)
// for W = 16, 2 ((k >> 1) & 1) + 4 ((k >> 3) & 1) for W = 8 and 2 ((k >> 3) & 1)
// for W = 4, which puts the eight k rows that a cycle of a transposing read
// takes two units of on distinct banks.  B as N x K is two halves of the
// tile's rows of four units, unit c of row r at 4 r + (c ^ 2 ((r >> 2) & 1)).  The
// halves may come from two matrices: a gated product's tile is the gate's
// columns and the up projection's same columns, so that a wavefront has both
// sums of its elements.  A as M x K is staged two stages at a time, whole
// 128-byte lines: rows of eight units, unit c of row r at 8 r + (c ^ ((r >> 1) & 7)).
//
// Pipeline.  Loads run D stages ahead: 3, and 7 on the 64 x 64 tile, whose
// stages are shorter.  B has D + 1 stage buffers, A as K x M too, A as M x K
// (D + 3) / 2 buffers of two stages.  During stage t the fragments of stage
// t + 1 are read and the loads of B stage t + D and A stage t + D (half of
// pair (t + D + 1) / 2) issued, spread between the MFMAs.  Each stage begins
// with a wait for this wavefront's loads of stage t + 1 and a barrier: then all
// of that stage has landed, and the buffers that are refilled were last read by
// fragments that every wavefront has since consumed.
//
// Bound by the matrix cores where there are tiles for every compute unit; the
// smaller tiles by LDS reads, 64, 96, 128, 192 and 256 bytes a cycle and
// compute unit of its 128 if the matrix cores never waited.
#include "common.h"
#include "lds_dma.h"
#include "linear.h"

namespace dgor {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) shortx4 lds_shortx4;

struct OpHalf : Half16 {
    static __device__ __forceinline__ floatx4 mfma(halfx8 a, halfx8 b, floatx4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
struct OpBrain : Brain16 {
    static __device__ __forceinline__ floatx4 mfma(halfx8 a, halfx8 b, floatx4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
};

constexpr uint32_t kOutside = 0x80000000u;   // a lane offset past every descriptor's range

template <int W>
__device__ __forceinline__ int row_swizzle(int k)
{
    return W == 16 ? 2 * (k & 3) + 8 * ((k >> 3) & 1)
                   : (W == 8 ? 2 * ((k >> 1) & 1) + 4 * ((k >> 3) & 1) : 2 * ((k >> 3) & 1));
}

// Descriptor range in bytes of `rows` rows of `cols` elements in whole units:
// what is past it reads as zero.
__device__ __forceinline__ int range_of(int rows, int cols, int ld)
{
    return rows <= 0 || cols <= 0
               ? 0
               : (int)(((uint32_t)(rows - 1) * (uint32_t)ld + ((uint32_t)(cols + 7) & ~7u)) * 2u);
}

// Stages that a load is ahead of its fragments' stage, and the ring's bytes.
constexpr int ring_ahead(int bm) { return bm == 64 ? 7 : 3; }
constexpr int ring_a_bytes(int bm, bool ta)
{
    const int d = ring_ahead(bm), stage = 32 * bm * 2;
    return ta ? (d + 1) * stage : ((d + 1) / 2 + 1) * 2 * stage;
}
constexpr int ring_bytes(int bm, int bn, bool ta) { return ring_a_bytes(bm, ta) + (ring_ahead(bm) + 1) * 32 * bn * 2; }

// Tile `bid` (of both batches) and part `part` of a product, by 256 threads.
template <class Op, int BM, int BN, bool TA, bool TB, bool GATED>
__device__ __forceinline__ void ring_tile(const Product &p, uint8_t *lds, int bid, int part)
{
    constexpr int BK = 32;
    constexpr int HM = BM / 2, HN = BN / 2;        // a wavefront's part of the tile,
    constexpr int FA = HM / 16, FB = HN / 16;      // and its 16-wide blocks
    constexpr int WA = HM / 8, WB = HN / 8;        // units of a half's k row
    constexpr int LPA = BM / 64, LPB = BN / 64;    // a wavefront's loads of each operand and stage
    constexpr int HALF_A = BK * HM * 2, HALF_B = BK * HN * 2, STAGE_A = 2 * HALF_A, STAGE_B = 2 * HALF_B;
    constexpr int PAIR = 2 * STAGE_A;
    constexpr int D = ring_ahead(BM), A_PAIRS = (D + 1) / 2 + 1;
    constexpr int A_BYTES = ring_a_bytes(BM, TA), LDS_BYTES = ring_bytes(BM, BN, TA);
    constexpr int FT = GATED ? HN : BN;            // output columns of a tile
    const uint32_t ring = lds_address(lds);

    const int per = p.tiles_m * p.tiles_n;
    const int batch = bid >= per ? 1 : 0;
    int tm, tn;
    dgor_tile_of_block(bid - batch * per, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    const int m0 = tm * BM, n0 = tn * FT;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int M = p.M, N = p.N, K = p.K, lda = p.lda, ldb = p.ldb;
    // stages of 32 k; of several segments each has a whole number of pairs
    const int seg_stages = 2 * ((K + 2 * BK - 1) / (2 * BK));
    const int total = p.nseg > 1 ? p.nseg * seg_stages : (K + BK - 1) / BK;
    const int s0 = p.splits > 1 ? part * p.chunk * 2 : 0;
    const int steps = (p.splits > 1 ? min(s0 + p.chunk * 2, total) : total) - s0;

    // ---- loads.  Wavefronts 0 and 1 fill half 0 of a stage, 2 and 3 half 1.
    const int lhalf = wave >> 1, alid0 = LPA * (wave & 1), blid0 = LPB * (wave & 1);
    const int bcol = GATED ? n0 : n0 + HN * lhalf;            // first column of this wavefront's half of B
    const int b_left = N - bcol;
    // the batch's segments, and the one that the sum begins in
    const int pairs_a = batch * p.nseg, pairs_b = GATED ? lhalf : pairs_a;
    const int seg0 = p.nseg > 1 ? s0 / seg_stages : 0;
    uint32_t b_off[LPB];
    const int b_kc = 8 * ((lane & 3) ^ (2 * ((lane >> 4) & 1)));
#pragma unroll
    for (int q = 0; q < LPB; ++q) {
        if (TB) {
            b_off[q] = (uint32_t)((16 * (blid0 + q) + (lane >> 2)) * ldb + b_kc) * 2u;
        } else {
            const int k = (64 / WB) * (blid0 + q) + lane / WB, u = (lane % WB) ^ row_swizzle<WB>(k);
            b_off[q] = 8 * u < b_left ? (uint32_t)(k * ldb + 8 * u) * 2u : kOutside;
        }
    }
    const uint32_t lds_b = ring + (uint32_t)(A_BYTES + lhalf * HALF_B + blid0 * 1024);
    struct Loads {
        intx4 r;
        int k_left;
        uint32_t dst;
    };
    // Where the next stage of an operand begins, how much of k is left there,
    // and how many stages until the next segment.  Kept and advanced rather
    // than found anew: a stage's scalar work is between its first MFMAs.
    struct Stream {
        const uint16_t *p;
        int k_left, until, seg;
        uint32_t dst;
    };
    const int k_first = BK * (s0 - seg0 * seg_stages);
    // stages of segment `seg` from its stage `gone` on; the last has no end, its
    // loads past k read zeros
    auto stages_of = [&](int seg, int gone) { return seg + 1 < p.nseg ? seg_stages - gone : 0x7fffffff; };
    const int until = stages_of(seg0, s0 - seg0 * seg_stages);
    const size_t b_row = TB ? (size_t)bcol * ldb : (size_t)bcol;
    const size_t b_step = TB ? 1 : (size_t)ldb;
    Stream bs{p.B.of(pairs_b + seg0, p.terms) + b_row + k_first * b_step, K - k_first, until, seg0, 0};
    auto b_loads = [&]() {
        Loads L;
        L.k_left = bs.k_left;
        L.r = rsrc_words(bs.p, 0);
        if (TB)
            L.r.z = L.k_left <= 0 ? 0 : (b_left >= HN ? 0x7fffffff : range_of(b_left, L.k_left, ldb));
        else
            L.r.z = L.k_left >= BK ? 0x7fffffff : range_of(L.k_left, b_left, ldb);
        L.dst = lds_b + bs.dst;
        bs.dst = (bs.dst + STAGE_B) & (uint32_t)((D + 1) * STAGE_B - 1);   // D + 1 is a power of two
        bs.p += BK * b_step;
        bs.k_left -= BK;
        if (--bs.until == 0)
            bs = Stream{p.B.of(pairs_b + bs.seg + 1, p.terms) + b_row, K, stages_of(bs.seg + 1, 0), bs.seg + 1, bs.dst};
        return L;
    };
    auto load_b = [&](const Loads &L, int q) {
        load_to_lds(L.r, L.dst + (uint32_t)(q * 1024), TB && b_kc >= L.k_left ? kOutside : b_off[q]);
    };
    // A as M x K: a wavefront loads a quarter of the tile's rows, eight a load
    uint32_t a_off[TA ? LPA : 2];
    int a_kc[2] = {0, 0};
    const int arow = TA ? m0 + HM * lhalf : m0;
    const int a_left = M - arow;
#pragma unroll
    for (int j = 0; j < (TA ? LPA : 2); ++j) {
        if (TA) {
            const int k = (64 / WA) * (alid0 + j) + lane / WA, u = (lane % WA) ^ row_swizzle<WA>(k);
            a_off[j] = 8 * u < a_left ? (uint32_t)(k * lda + 8 * u) * 2u : kOutside;
        } else {
            const int r = (HM / 2) * wave + 8 * j + (lane >> 3);
            const int c = (lane & 7) ^ ((4 * j + (lane >> 4)) & 7);
            a_off[j] = (uint32_t)(r * lda + 8 * c) * 2u;
            a_kc[j] = 8 * c;
        }
    }
    const uint32_t a_row16 = (uint32_t)(16 * lda) * 2u;
    const uint32_t lds_a = ring + (uint32_t)(TA ? lhalf * HALF_A + alid0 * 1024 : 2 * LPA * wave * 1024);
    // loads of the next A stage (A as K x M) or pair of stages
    constexpr int A_DEEP = TA ? BK : 2 * BK;
    const size_t a_row = TA ? (size_t)arow : (size_t)m0 * lda;
    const size_t a_step = TA ? (size_t)lda : 1;
    Stream as{p.A.of(pairs_a + seg0, p.terms) + a_row + k_first * a_step, K - k_first, until, seg0, 0};
    auto a_loads = [&]() {
        Loads L;
        L.k_left = as.k_left;
        L.r = rsrc_words(as.p, 0);
        if (TA)
            L.r.z = L.k_left >= BK ? 0x7fffffff : range_of(L.k_left, a_left, lda);
        else
            L.r.z = L.k_left <= 0 ? 0 : (a_left >= BM ? 0x7fffffff : range_of(a_left, L.k_left, lda));
        L.dst = lds_a + as.dst;
        if (TA)
            as.dst = (as.dst + STAGE_A) & (uint32_t)((D + 1) * STAGE_A - 1);
        else
            as.dst = as.dst == (uint32_t)((A_PAIRS - 1) * PAIR) ? 0u : as.dst + PAIR;
        as.p += A_DEEP * a_step;
        as.k_left -= A_DEEP;
        as.until -= A_DEEP / BK;
        if (as.until == 0)
            as = Stream{p.A.of(pairs_a + as.seg + 1, p.terms) + a_row, K, stages_of(as.seg + 1, 0), as.seg + 1, as.dst};
        return L;
    };
    auto load_a = [&](const Loads &L, int j) {
        uint32_t off;
        if (TA)
            off = a_off[j];
        else
            off = a_kc[j & 1] >= L.k_left ? kOutside : a_off[j & 1] + (uint32_t)(j >> 1) * a_row16;
        load_to_lds(L.r, L.dst + (uint32_t)(j * 1024), off);
    };

    // ---- fragments.  Lane (g, s) = (lane / 16, lane % 16).
    const int s16 = lane & 15, g = lane >> 4;
    const int wrow = (wave >> 1) * HM;
    // k rows 8 g + s / 4 and four further: both have this swizzle
    const int kr = 8 * g + (s16 >> 2), a_x = row_swizzle<WA>(kr), b_x = row_swizzle<WB>(kr);
    constexpr int FU = GATED ? FB / 2 : FB;        // distinct column blocks of B
    uint32_t b_unit[TB ? 1 : FU], a_unit[TA ? FA : 1];
    if (!TB)
#pragma unroll
        for (int j = 0; j < FU; ++j)
            b_unit[TB ? 0 : j] =
                (uint32_t)(((2 * ((GATED ? (wave & 1) * FU : 0) + j) + ((s16 & 3) >> 1)) ^ b_x) * 16);
    if (TA)
#pragma unroll
        for (int i = 0; i < FA; ++i)
            a_unit[TA ? i : 0] = (uint32_t)(((2 * i + ((s16 & 3) >> 1)) ^ a_x) * 16);
    const uint32_t kc_lane = (uint32_t)(s16 * 64 + ((g ^ (2 * ((s16 >> 2) & 1))) * 16));
    const uint32_t b_lane = (uint32_t)A_BYTES + (TB ? kc_lane : (uint32_t)(kr * (HN * 2) + 8 * (s16 & 1))) +
                            (GATED ? (TB ? (uint32_t)((wave & 1) * FU * 1024) : 0u) : (uint32_t)((wave & 1) * HALF_B));
    const uint32_t a_lane = TA ? (uint32_t)(kr * (HM * 2) + 8 * (s16 & 1) + (wave >> 1) * HALF_A)
                               : (uint32_t)((wrow + s16) * 128) | (uint32_t)((g ^ ((s16 >> 1) & 7)) * 16);
    auto transposed = [&](uint32_t at, int row) -> halfx8 {   // row: bytes of a k row
        const uint8_t *q = lds + at;
        const shortx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4 *)q);
        const shortx4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4 *)(q + 4 * row));
        return __builtin_bit_cast(halfx8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    struct Source {
        uint32_t a;      // byte offset of the stage's A buffer
        int odd;         // second stage of its pair (A as M x K)
        uint32_t b;      // and of its B buffer
    };
    auto read_a = [&](const Source &S, int i) -> halfx8 {
        if (TA)
            return transposed(a_lane + S.a + a_unit[TA ? i : 0], HM * 2);
        return *reinterpret_cast<const halfx8 *>(lds + ((a_lane ^ (uint32_t)(64 * S.odd)) + S.a + (uint32_t)(i * 2048)));
    };
    auto read_b = [&](const Source &S, int j) -> halfx8 {
        const uint32_t at = b_lane + S.b + (GATED ? (uint32_t)((j / FU) * HALF_B) : 0u);
        if (TB)
            return *reinterpret_cast<const halfx8 *>(lds + at + (uint32_t)((j % FU) * 1024));
        return transposed(at + b_unit[TB ? 0 : j % FU], HN * 2);
    };
    // A block 0, the B blocks, then the other A blocks: as the MFMAs want them
    auto fread = [&](const Source &S, int r, halfx8 *fa, halfx8 *fb) {
        if (r == 0 || r > FB)
            fa[r == 0 ? 0 : r - FB] = read_a(S, r == 0 ? 0 : r - FB);
        else
            fb[r - 1] = read_b(S, r - 1);
    };

    floatx4 acc[FA][FB];
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                asm("v_accvgpr_write_b32 %0, 0" : "=a"(acc[i][j][r]));   // keeps the array in the accumulators

    // One stage: its MFMAs from (ca, cb), the next stage's fragment reads after
    // the first of them, then its loads.  par: the stage within its pair; half
    // a pair of A (as M x K) is loaded in each.
    Loads LA, LB;
    auto stage = [&](int par, const Source &S, halfx8 *ca, halfx8 *cb, halfx8 *na, halfx8 *nb) {
        constexpr int MFMAS = FA * FB, READS = FA + FB, LOADS = LPA + LPB;
        // a load every EVERY MFMAs: after the reads, or (too few MFMAs after
        // them; the 64 x 64 tile is 12% faster so) among them
        constexpr int FIRST = MFMAS - READS >= LOADS ? READS : 2, EVERY = (MFMAS - FIRST) / LOADS;
        auto issue = [&](int ld) {
            if (ld < LPB)
                load_b(LB, ld);
            else if (ld < LOADS)
                load_a(LA, (TA ? 0 : LPA * par) + ld - LPB);
        };
#pragma unroll
        for (int m = 0; m < FA * FB; ++m) {
            const int i = m / FB, j = m % FB;
            acc[i][j] = Op::mfma(ca[i], cb[j], acc[i][j]);
            if (m < READS)
                fread(S, m, na, nb);
            if (m == 0)
                LB = b_loads();
            if (m == 1 && (TA || par == 0))
                LA = a_loads();
            if (m >= FIRST && (m - FIRST) % EVERY == EVERY - 1)
                issue((m - FIRST) / EVERY);
            // keep this order: the compiler would otherwise cluster the reads
            // and loads, and move MFMAs across the barrier
            __builtin_amdgcn_sched_barrier(0);
        }
        static_assert((MFMAS - FIRST) / EVERY >= LOADS && READS <= MFMAS, "all issued");
    };
    auto next_pair = [](uint32_t b) { return b == (uint32_t)((A_PAIRS - 1) * PAIR) ? 0u : b + PAIR; };
    auto source = [&](int t, uint32_t pair) {   // stage t's buffers
        const uint32_t b = (uint32_t)((t & D) * STAGE_B);
        return TA ? Source{(uint32_t)((t & D) * STAGE_A), 0, b} : Source{pair, t & 1, b};
    };

    halfx8 fa0[FA], fa1[FA], fb0[FB], fb1[FB];
    // in the order of their stages: A 0 (or pair 0), B 0; B 1; pair 1, B 2; ...
#pragma unroll
    for (int st = 0; st < D; ++st) {
        if (TA || st % 2 == 0) {
            LA = a_loads();
#pragma unroll
            for (int j = 0; j < (TA ? LPA : 2 * LPA); ++j)
                load_a(LA, j);
        }
        LB = b_loads();
#pragma unroll
        for (int q = 0; q < LPB; ++q)
            load_b(LB, q);
    }
    // A and B of stage 0 have landed
    __builtin_amdgcn_s_waitcnt(wait_vmcnt((D - 1) * (LPA + LPB)));
    __builtin_amdgcn_s_barrier();
    {
        const Source S = source(0, 0);
#pragma unroll
        for (int r = 0; r < FA + FB; ++r)
            fread(S, r, fa0, fb0);
    }
    // Before stage t: B stage t + 1 and the A it reads have landed.  Loads are
    // in the order of their stages, each stage's B first; an even stage's next
    // stage is of the pair it already reads.
    auto wait = [&](int par) {
        if (!TA && par == 0)
            __builtin_amdgcn_s_waitcnt(wait_vmcnt_lgkm0((D - 2) * (LPA + LPB) + LPA));
        else
            __builtin_amdgcn_s_waitcnt(wait_vmcnt_lgkm0((D - 2) * (LPA + LPB)));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    uint32_t pa = 0;   // the pair's buffer
    for (int t = 0; t < steps; t += 2) {
        const uint32_t pa1 = next_pair(pa);
        wait(0);
        stage(0, source(t + 1, pa), fa0, fb0, fa1, fb1);
        if (t + 1 < steps) {
            wait(1);
            stage(1, source(t + 2, pa1), fa1, fb1, fa0, fb0);
        }
        pa = pa1;
    }
    // no load may still be writing LDS, nor a wavefront reading the ring
    __builtin_amdgcn_s_waitcnt(wait_vmcnt_lgkm0(0));
    __builtin_amdgcn_s_barrier();
    dgor_acc_hazard_wait();

    // Epilogue: 32 rows at a time through the wavefront's own part of LDS, so
    // that a lane holds eight neighbouring columns of one row.  Rows are padded
    // by 16 bytes, which puts the 64 lanes of each write on distinct banks.
    constexpr int ROW = HN + 4;                                   // floats
    constexpr int COLS = GATED ? HN / 2 : HN, LANES = COLS / 8;
    static_assert(4 * 32 * ROW * 4 <= LDS_BYTES, "the epilogue uses the ring's LDS");
    float *w = reinterpret_cast<float *>(lds) + wave * 32 * ROW;
    const int c0 = n0 + (wave & 1) * COLS;
    Epilogue e = p.e;
    if (batch)
        e.Y = p.Y1;
    // a lane keeps its columns through all rounds, every STEP-th row of each
    constexpr int STEP = 64 / LANES, TURNS = 32 / STEP, TOGETHER = TURNS < 2 ? 1 : 2;
    const int r0 = lane / LANES, c = 8 * (lane % LANES), col = c0 + c, cols = N - col;
    const bool mine = cols > 0, whole = n0 + FT <= N;
    float bias[8] = {};
    if (!GATED && mine && p.splits <= 1)
        load_bias<Op>(e, col, cols, bias);
    // one copy of the code behind the accumulators: unrolled, its first run
    // waits for instructions longer than it works (256 x 256 tile: 10 us)
#pragma unroll 1
    for (int round = 0; round < FA / 2; ++round) {
#pragma unroll
        for (int k = 0; k < FA / 2; ++k)
            if (round == k) {
#pragma unroll
                for (int ii = 0; ii < 2; ++ii)
#pragma unroll
                    for (int j = 0; j < FB; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            w[(16 * ii + 4 * g + r) * ROW + 16 * j + s16] = dgor_acc_read(acc[2 * k + ii][j][r]);
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        // the round's rows, TOGETHER at a time, to take(first row, v, u)
        auto rows = [&](auto take) {
#pragma unroll 1
            for (int q0 = 0; q0 < TURNS; q0 += TOGETHER) {
                const int lr = r0 + STEP * q0, row = m0 + wrow + 32 * round + lr;
                if (!mine || row >= M)
                    break;
                float v[TOGETHER][8], u[TOGETHER][8];
#pragma unroll
                for (int q = 0; q < TOGETHER; ++q)
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        v[q][x] = w[(lr + STEP * q) * ROW + c + x];
                        u[q][x] = GATED ? w[(lr + STEP * q) * ROW + COLS + c + x] : 0.f;
                    }
                take(row, v, u);
            }
        };
        typedef float Rows[TOGETHER][8];
        if (p.splits > 1) {
            rows([&](int row, Rows &v, Rows &u) {
                const int ld = part_stride(p);
                float *to = p.part + ((size_t)batch * p.splits + part) * part_size(p) + (size_t)row * ld + col;
#pragma unroll
                for (int q = 0; q < TOGETHER; ++q)
                    if (row + STEP * q < M) {
                        store8_f32(to + (size_t)(STEP * q) * ld, 8, v[q]);
                        if (GATED)
                            store8_f32(to + p.splits * part_size(p) + (size_t)(STEP * q) * ld, 8, u[q]);
                    }
            });
        } else if (!whole) {
            rows([&](int row, Rows &v, Rows &u) {
                emit_rows<Op, GATED, false, kAnyActivation, TOGETHER>(e, row, STEP, M, col, cols, v, u, bias);
            });
        } else {
            // a copy for each activation: the branch is taken once a round,
            // and the values stay in their registers
            switch (e.act) {
#define DGOR_ROWS(A)                                                                              \
    rows([&](int row, Rows &v, Rows &u) {                                                         \
        emit_rows<Op, GATED, true, A, TOGETHER>(e, row, STEP, M, col, 8, v, u, bias);             \
    });                                                                                           \
    break
            case GEMM_ACT_RELU: DGOR_ROWS(GEMM_ACT_RELU);
            case GEMM_ACT_GELU: DGOR_ROWS(GEMM_ACT_GELU);
            case GEMM_ACT_GELU_TANH: DGOR_ROWS(GEMM_ACT_GELU_TANH);
            case GEMM_ACT_SILU: DGOR_ROWS(GEMM_ACT_SILU);
            default: DGOR_ROWS(GEMM_ACT_NONE);
#undef DGOR_ROWS
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

template <class Op, int BM, int BN, bool TA, bool TB, bool GATED>
__global__ __launch_bounds__(256) void linear_ring_kernel(Product p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[ring_bytes(BM, BN, TA)];
    ring_tile<Op, BM, BN, TA, TB, GATED>(p, lds, (int)blockIdx.x, (int)blockIdx.y);
}

// Both products of a backward pass in one launch: first the workgroups of the
// weight's gradient w, then those of the input's gradient x.
template <class Op, int BM, int BN, bool TB>
__global__ __launch_bounds__(256) void linear_ring_pair_kernel(Product w, Product x, int w_groups)
{
    constexpr int A = ring_bytes(BM, BN, true), B = ring_bytes(BM, BN, false);
    __shared__ __attribute__((aligned(1024))) uint8_t lds[A > B ? A : B];
    const bool first = (int)blockIdx.x < w_groups;
    const Product &p = first ? w : x;
    const int id = (int)blockIdx.x - (first ? 0 : w_groups), per = p.tiles_m * p.tiles_n * p.nbatch;
    if (first)
        ring_tile<Op, BM, BN, true, false, false>(w, lds, id % per, id / per);
    else
        ring_tile<Op, BM, BN, false, TB, false>(x, lds, id % per, id / per);
}

template <class Op, int BM, int BN>
hipError_t launch_pair_as(const Product &w, const Product &x, hipStream_t s)
{
    const int nw = w.tiles_m * w.tiles_n * w.nbatch * (w.splits > 1 ? w.splits : 1);
    const int nx = x.tiles_m * x.tiles_n * (x.splits > 1 ? x.splits : 1);
    const auto kernel =
        x.trans_b ? linear_ring_pair_kernel<Op, BM, BN, true> : linear_ring_pair_kernel<Op, BM, BN, false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(nw + nx)), dim3(256), 0, s, w, x, nw);
    return hipGetLastError();
}

void lay_out(Product &p, RingTile tile)
{
    const int bm = ring_tile_m(tile), bn = ring_tile_n(tile), ft = p.gated ? bn / 2 : bn;
    p.tiles_m = (p.M + bm - 1) / bm;
    p.tiles_n = (p.N + ft - 1) / ft;
    p.group_m = 4;
}

template <class Op, int BM, int BN>
hipError_t launch_ring_as(const Product &p, hipStream_t s)
{
    const dim3 grid((unsigned)(p.tiles_m * p.tiles_n * p.nbatch), (unsigned)(p.splits > 1 ? p.splits : 1));
    if (p.gated) {
        if (p.trans_b)
            hipLaunchKernelGGL((linear_ring_kernel<Op, BM, BN, false, true, true>), grid, dim3(256), 0, s, p);
        else
            hipLaunchKernelGGL((linear_ring_kernel<Op, BM, BN, false, false, true>), grid, dim3(256), 0, s, p);
    } else if (p.trans_a) {
        hipLaunchKernelGGL((linear_ring_kernel<Op, BM, BN, true, false, false>), grid, dim3(256), 0, s, p);
    } else if (p.trans_b) {
        hipLaunchKernelGGL((linear_ring_kernel<Op, BM, BN, false, true, false>), grid, dim3(256), 0, s, p);
    } else {
        hipLaunchKernelGGL((linear_ring_kernel<Op, BM, BN, false, false, false>), grid, dim3(256), 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_ring(const Product &q, RingTile tile, hipStream_t s)
{
    Product p = q;
    if (p.trans_a && p.trans_b)
        return hipErrorInvalidValue;
    lay_out(p, tile);
    switch (tile) {
    case kRing256: return p.bf16 ? launch_ring_as<OpBrain, 256, 256>(p, s) : launch_ring_as<OpHalf, 256, 256>(p, s);
    case kRing256x128:
        return p.bf16 ? launch_ring_as<OpBrain, 256, 128>(p, s) : launch_ring_as<OpHalf, 256, 128>(p, s);
    case kRing128: return p.bf16 ? launch_ring_as<OpBrain, 128, 128>(p, s) : launch_ring_as<OpHalf, 128, 128>(p, s);
    case kRing128x64: return p.bf16 ? launch_ring_as<OpBrain, 128, 64>(p, s) : launch_ring_as<OpHalf, 128, 64>(p, s);
    case kRing64: return p.bf16 ? launch_ring_as<OpBrain, 64, 64>(p, s) : launch_ring_as<OpHalf, 64, 64>(p, s);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_linear_ring_pair(const Product &weight, const Product &input, RingTile tile, hipStream_t s)
{
    Product w = weight, x = input;
    if (!w.trans_a || w.trans_b || x.trans_a || w.gated || x.gated || x.nbatch != 1)
        return hipErrorInvalidValue;
    lay_out(w, tile);
    lay_out(x, tile);
    switch (tile) {
    case kRing128:
        return w.bf16 ? launch_pair_as<OpBrain, 128, 128>(w, x, s) : launch_pair_as<OpHalf, 128, 128>(w, x, s);
    case kRing128x64:
        return w.bf16 ? launch_pair_as<OpBrain, 128, 64>(w, x, s) : launch_pair_as<OpHalf, 128, 64>(w, x, s);
    case kRing64: return w.bf16 ? launch_pair_as<OpBrain, 64, 64>(w, x, s) : launch_pair_as<OpHalf, 64, 64>(w, x, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace dgor
