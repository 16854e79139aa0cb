// The dense-layer products of 16-byte aligned operands: the main loop of
// ring.h on tiles of 256 x 256, 256 x 128, 128 x 128, 128 x 64 and 64 x 64, and
// the epilogue of epilogue.h on whole rows.
#include "ring.h"

namespace dgor {
namespace {

using namespace ring;

// Tile `bid` (of both batches) and part `part` of a product, by 256 threads.
template <class Op, int BM, int BN, bool TA, bool TB, bool GATED>
__device__ __forceinline__ void ring_tile(const Product &p, uint8_t *lds, int bid, int part)
{
    constexpr int HM = BM / 2, HN = BN / 2;        // a wavefront's part of the tile,
    constexpr int FA = HM / 16, FB = HN / 16;      // and its 16-wide blocks
    constexpr int LDS_BYTES = ring_bytes(BM, BN, TA);
    constexpr int FT = GATED ? HN : BN;            // output columns of a tile
    const int per = p.tiles_m * p.tiles_n;
    const int batch = bid >= per ? 1 : 0;
    int tm, tn;
    dgor_tile_of_block(bid - batch * per, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    floatx4 acc[FA][FB];
    ring_sum<Op, BM, BN, TA, TB, GATED>(p, lds, tm, tn, batch, part, acc);
    const int m0 = tm * BM, n0 = tn * FT, M = p.M, N = p.N;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wrow = (wave >> 1) * HM;

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
        stage_rows(acc, round, w, ROW, lane);
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
