// The dense-layer product for operands that neither the rings nor the few-row
// kernel take (addresses off 16 bytes under strides on it, strides of 2^22 and
// more, matrices smaller than a 16-byte unit): 64 x 64 tiles staged through
// registers into LDS, FP32 sums on v_mfma_f32_16x16x32, and the epilogue of
// epilogue.h on whole rows.  Any size, stride and alignment; written to be
// short rather than fast.
//
// Both operands may be k-contiguous (A as M x K, B as N x K) or k-strided (A
// as K x M, B as K x N).  A stage is 64 k.  In 16-byte units (8 elements):
//   k-contiguous: rows of 8 units, unit c of row r at 8 r + (c ^ ((r >> 1) & 7));
//     a fragment is one 128-bit read of a row;
//   k-strided: 64 k rows of W = 8 units, unit u of row k at W k + (u ^ x(k)),
//     x(k) = 2 ((k >> 1) & 1) + 4 ((k >> 3) & 1): the eight k rows that a cycle
//     of a transposing read takes two units of fall on distinct units modulo
//     16.
// Global loads take 16 bytes at any element address; only the units that an
// edge of the matrix cuts are read element by element.
#include "common.h"
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

// Eight elements of row r from column c of a rows x cols matrix, zero outside.
__device__ __forceinline__ u32x4 load_unit(const uint16_t *p, size_t ld, int r, int rows, int c, int cols)
{
    if (r >= rows || c >= cols)
        return u32x4{0u, 0u, 0u, 0u};
    return load8_16(p + (size_t)r * ld + c, cols - c);
}

__device__ __forceinline__ int strided_swizzle(int k) { return 2 * ((k >> 1) & 1) + 4 * ((k >> 3) & 1); }

template <class Op, bool TA, bool TB, bool GATED>
__global__ __launch_bounds__(256) void linear_tile_kernel(Product p)
{
    constexpr int BT = kTile, BK = kStageDepth;
    constexpr int W = BT / 8;                    // units of a k-strided row
    constexpr int UNITS = BT * BK / 8 / 256;     // units a thread loads of each operand and stage
    constexpr int FT = GATED ? BT / 2 : BT;      // output columns of a tile
    constexpr int WT = BT / 2, FM = WT / 16;     // a wavefront's square of the tile, in rows and 16-row blocks
    constexpr int OPERAND = BT * BK * 2;         // bytes
    static_assert(UNITS * 256 * 8 == BT * BK, "units must divide");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * OPERAND];   // two stages of A and B

    const int per = p.tiles_m * p.tiles_n;
    const int batch = blockIdx.x >= (unsigned)per ? 1 : 0;
    int tm, tn;
    dgor_tile_of_block((int)blockIdx.x - batch * per, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    const int m0 = tm * BT, n0 = tn * FT;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = (wave >> 1) * WT, wc = (wave & 1) * WT;
    const int M = p.M, N = p.N, K = p.K;
    const int per_seg = (K + BK - 1) / BK;
    const int t0 = p.splits > 1 ? (int)blockIdx.y * p.chunk : 0;
    const int t1 = p.splits > 1 ? min(t0 + p.chunk, p.nseg * per_seg) : p.nseg * per_seg;

    // Local column j of the tile's B: the feature for a gated product, whose
    // tile holds, for each half of its columns, the gate's and then the up
    // projection's same features (so one wavefront has both sums of each).
    auto b_col = [&](int j, int &which) {
        which = GATED ? (j / (WT / 2)) & 1 : 0;
        return n0 + (GATED ? (j / WT) * (WT / 2) + j % (WT / 2) : j);
    };
    u32x4 ra[UNITS], rb[UNITS];
    auto load_stage = [&](int t) {
        const int seg = p.nseg > 1 ? t / per_seg : 0, pair = batch * p.nseg + seg;
        const int k0 = (t - seg * per_seg) * BK;
        const uint16_t *A = p.A.of(pair, p.terms);
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            const int u = tid + 256 * i;
            if (TA)
                ra[i] = load_unit(A, p.lda, k0 + u / W, K, m0 + 8 * (u % W), M);
            else
                ra[i] = load_unit(A, p.lda, m0 + u / 8, M, k0 + 8 * (u % 8), K);
            int which;
            if (TB) {
                const int n = b_col(u / 8, which);
                rb[i] = load_unit(p.B.of(GATED ? which : pair, p.terms), p.ldb, n, N, k0 + 8 * (u % 8), K);
            } else {
                const int n = b_col(8 * (u % W), which);
                rb[i] = load_unit(p.B.of(GATED ? which : pair, p.terms), p.ldb, k0 + u / W, K, n, N);
            }
        }
    };
    auto slot = [&](bool strided, int u) {
        return strided ? W * (u / W) + ((u % W) ^ strided_swizzle(u / W)) : 8 * (u / 8) + ((u % 8) ^ ((u / 16) & 7));
    };
    auto store_stage = [&](int buf) {
        uint8_t *base = lds + buf * 2 * OPERAND;
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            const int u = tid + 256 * i;
            *reinterpret_cast<u32x4 *>(base + 16 * slot(TA, u)) = ra[i];
            *reinterpret_cast<u32x4 *>(base + OPERAND + 16 * slot(!TB, u)) = rb[i];
        }
    };
    const int s16 = lane & 15, g = lane >> 4;
    // fragment of the 16 rows (columns of B) from `at`, k 32 half + 8 g .. + 7
    auto fragment = [&](const uint8_t *op, bool strided, int at, int half) -> halfx8 {
        if (!strided) {
            const int r = at + s16;
            return *reinterpret_cast<const halfx8 *>(op + 16 * (8 * r + ((4 * half + g) ^ ((r >> 1) & 7))));
        }
        const int k = 32 * half + 8 * g + (s16 >> 2);
        const int u = at / 8 + ((s16 & 3) >> 1);
        const uint8_t *lo = op + 16 * (W * k + (u ^ strided_swizzle(k))) + 8 * (s16 & 1);
        const int k4 = k + 4;
        const uint8_t *hi = op + 16 * (W * k4 + (u ^ strided_swizzle(k4))) + 8 * (s16 & 1);
        const shortx4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4 *)lo);
        const shortx4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4 *)hi);
        return __builtin_bit_cast(halfx8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    };

    floatx4 acc[FM][FM];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
            acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    if (t0 < t1) {
        load_stage(t0);
        store_stage(0);
    }
    __syncthreads();
    for (int t = t0; t < t1; ++t) {
        const uint8_t *base = lds + ((t - t0) & 1) * 2 * OPERAND;
        if (t + 1 < t1)
            load_stage(t + 1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            halfx8 a[FM], b[FM];
#pragma unroll
            for (int i = 0; i < FM; ++i)
                a[i] = fragment(base, TA, wr + 16 * i, half);
#pragma unroll
            for (int j = 0; j < FM; ++j)
                b[j] = fragment(base + OPERAND, !TB, wc + 16 * j, half);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    acc[i][j] = Op::mfma(a[i], b[j], acc[i][j]);
        }
        if (t + 1 < t1) {
            store_stage((t - t0 + 1) & 1);   // last read one stage ago, before that stage's barrier
            __syncthreads();
        }
    }
    __syncthreads();

    // Epilogue: each wavefront's rows go through its own part of LDS, 16 at a
    // time, so that a lane holds eight neighbouring columns of one row.
    constexpr int ROW = WT + 4;   // floats; the padding spreads the four-row groups over the banks
    constexpr int COLS = GATED ? WT / 2 : WT, LANES = COLS / 8;
    float *w = reinterpret_cast<float *>(lds) + wave * 16 * ROW;
    const int c0 = n0 + (GATED ? wc / 2 : wc);
    Epilogue e = p.e;
    if (batch)
        e.Y = p.Y1;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FM; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                w[(4 * g + r) * ROW + 16 * j + s16] = acc[i][j][r];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < (16 * LANES + 63) / 64; ++q) {
            const int id = lane + 64 * q, r = id / LANES, c = 8 * (id % LANES);
            const int row = m0 + wr + 16 * i + r, col = c0 + c;
            if (r < 16 && row < M && col < N) {
                float v[8], u[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    v[x] = w[r * ROW + c + x];
                    u[x] = GATED ? w[r * ROW + COLS + c + x] : 0.f;
                }
                if (p.splits > 1) {
                    float *part = p.part + ((size_t)batch * p.splits + blockIdx.y) * part_size(p) +
                                  (size_t)row * part_stride(p) + col;
                    store8_f32(part, 8, v);
                    if (GATED)
                        store8_f32(part + p.splits * part_size(p), 8, u);
                } else {
                    emit8<Op, GATED>(e, row, col, N - col, v, u);
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// Adds the partial sums of a product that was split over k, in split order,
// eight neighbouring outputs a thread.
template <class Op, bool GATED>
__global__ __launch_bounds__(256) void linear_join_kernel(Product p)
{
    const int batch = blockIdx.y;
    const size_t size = part_size(p);
    const unsigned groups = (unsigned)(p.N + 7) / 8;
    const unsigned id = blockIdx.x * 256 + threadIdx.x;   // split products are small
    if (id >= (unsigned)p.M * groups)
        return;
    const int row = (int)(id / groups), col = 8 * (int)(id % groups), n = p.N - col;
    float v[8] = {}, u[8] = {};
    const float *q = p.part + (size_t)batch * p.splits * size + (size_t)row * part_stride(p) + col;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
        float t[8];
        load8_f32(q + s * size, 8, t);
#pragma unroll
        for (int x = 0; x < 8; ++x)
            v[x] += t[x];
        if (GATED) {
            load8_f32(q + (p.splits + s) * size, 8, t);
#pragma unroll
            for (int x = 0; x < 8; ++x)
                u[x] += t[x];
        }
    }
    Epilogue e = p.e;
    if (batch)
        e.Y = p.Y1;
    emit8<Op, GATED>(e, row, col, n, v, u);
}

template <class Op>
hipError_t launch_tile_as(const Product &p, hipStream_t s)
{
    const dim3 grid((unsigned)(p.tiles_m * p.tiles_n * p.nbatch), (unsigned)(p.splits > 1 ? p.splits : 1));
    if (p.gated) {
        if (p.trans_b)
            hipLaunchKernelGGL((linear_tile_kernel<Op, false, true, true>), grid, dim3(256), 0, s, p);
        else
            hipLaunchKernelGGL((linear_tile_kernel<Op, false, false, true>), grid, dim3(256), 0, s, p);
    } else if (p.trans_a) {
        hipLaunchKernelGGL((linear_tile_kernel<Op, true, false, false>), grid, dim3(256), 0, s, p);
    } else if (p.trans_b) {
        hipLaunchKernelGGL((linear_tile_kernel<Op, false, true, false>), grid, dim3(256), 0, s, p);
    } else {
        hipLaunchKernelGGL((linear_tile_kernel<Op, false, false, false>), grid, dim3(256), 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_tile(const Product &q, hipStream_t s)
{
    Product p = q;
    const int ft = p.gated ? kTile / 2 : kTile;
    p.tiles_m = (p.M + kTile - 1) / kTile;
    p.tiles_n = (p.N + ft - 1) / ft;
    p.group_m = 4;
    if (p.trans_a && p.trans_b)
        return hipErrorInvalidValue;
    return p.bf16 ? launch_tile_as<OpBrain>(p, s) : launch_tile_as<OpHalf>(p, s);
}

hipError_t launch_join(const Product &p, hipStream_t s)
{
    const size_t threads = (size_t)p.M * ((p.N + 7) / 8);
    const dim3 grid((unsigned)((threads + 255) / 256), (unsigned)p.nbatch);
    if (p.gated)
        hipLaunchKernelGGL((p.bf16 ? linear_join_kernel<OpBrain, true> : linear_join_kernel<OpHalf, true>), grid,
                           dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((p.bf16 ? linear_join_kernel<OpBrain, false> : linear_join_kernel<OpHalf, false>), grid,
                           dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace dgor
