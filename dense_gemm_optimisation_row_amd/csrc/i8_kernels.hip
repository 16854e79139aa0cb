// The products of int8 operands with a scale for each row of A and each column of
// B, Y = act(row[m] col[n] sum_k A[m][k] B[n][k] + bias[n]) + R, and the gated
// one of two matrices B.  Sums on v_mfma_i32_16x16x64_i8, exact in INT32; what
// follows them in FP32, rounded once.
//
// Both operands' rows run along k, so two k are one 16-bit element to the main
// loop of ring.h: its 32-deep stages hold 64 k, and a lane's 16 bytes are k
// 16 g .. 16 g + 15 of row s, which is what the instruction takes.  A K x N matrix
// is transposed into the workspace first.
//
// Large products are bound by the matrix cores, products of few rows by reading B.
#include <type_traits>

#include "i8.h"
#include "ring.h"

namespace dgor {
namespace {

using namespace ring;

typedef u32x4 u32x4_at1 __attribute__((aligned(1)));

struct OpInt8 {
    static __device__ __forceinline__ intx4 mfma(halfx8 a, halfx8 b, intx4 c)
    {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(intx4, a), __builtin_bit_cast(intx4, b), c, 0,
                                                     0, 0);
    }
};

// What a lane keeps for its eight columns, n of them inside the matrix.
template <bool GATED>
struct Columns {
    float scale[8], second[8];   // second: the up projection's scales, or the bias
    __device__ __forceinline__ void load(const I8Epilogue &e, int col, int n)
    {
        load8_f32(e.col + col, n, scale);
        const float *p = GATED ? e.up : e.bias;
        if (p)
            load8_f32(p + col, n, second);
        else
#pragma unroll
            for (int c = 0; c < 8; ++c)
                second[c] = 0.f;
    }
};

// Eight neighbouring outputs of each of the rows row, row + step, ... below M: v
// (and u, gated) the INT32 sums' bits.  The residual is read by the lane that
// writes the same elements of Y, so Y may be the residual itself.
template <bool GATED, bool WHOLE, int ACT, int ROWS>
__device__ __forceinline__ void emit_i8(const I8Epilogue &e, int row, int step, int M, int col, int inside,
                                        float (&v)[ROWS][8], const float (&u)[ROWS][8], const Columns<GATED> &k)
{
    const int n = WHOLE ? 8 : inside;
    float r[ROWS][8], s[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int at = row + i * step < M ? row + i * step : row;
        s[i] = e.row[at];
        if (!GATED && e.R)
            load8_of(e.fmt, e.R, (size_t)at * e.ldr + col, n, r[i]);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float z = (float)__float_as_int(v[i][c]) * s[i] * k.scale[c];
            if (GATED)
                v[i][c] = activate(ACT, z) * ((float)__float_as_int(u[i][c]) * s[i] * k.second[c]);
            else
                v[i][c] = activate(ACT, z + k.second[c]);
            if (!GATED && e.R)
                v[i][c] += r[i][c];
        }
        if (row + i * step < M)
            store8_of(e.fmt, e.Y, (size_t)(row + i * step) * e.ldy + col, n, v[i]);
    }
}

// emit with the activation as a constant: one uniform branch.
template <class F>
__device__ __forceinline__ void with_activation(int act, F f)
{
    switch (act) {
    case GEMM_ACT_RELU: f(std::integral_constant<int, GEMM_ACT_RELU>()); break;
    case GEMM_ACT_GELU: f(std::integral_constant<int, GEMM_ACT_GELU>()); break;
    case GEMM_ACT_GELU_TANH: f(std::integral_constant<int, GEMM_ACT_GELU_TANH>()); break;
    case GEMM_ACT_SILU: f(std::integral_constant<int, GEMM_ACT_SILU>()); break;
    default: f(std::integral_constant<int, GEMM_ACT_NONE>()); break;
    }
}

// ------------------------------------------------------------------ rings --

template <int BM, int BN, bool GATED>
__global__ __launch_bounds__(256) void i8_ring_kernel(Product p, I8Epilogue e)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[ring_bytes(BM, BN, false)];
    constexpr int HM = BM / 2, HN = BN / 2, FA = HM / 16, FB = HN / 16;
    constexpr int FT = GATED ? HN : BN;            // output columns of a tile
    int tm, tn;
    dgor_tile_of_block((int)blockIdx.x, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    const int part = (int)blockIdx.y;
    intx4 acc[FA][FB];
    ring_sum<OpInt8, BM, BN, false, true, GATED>(p, lds, tm, tn, 0, part, acc);

    // 32 rows at a time through the wavefront's own part of LDS, so that a lane
    // holds eight neighbouring columns of one row; rows are padded by 16 bytes,
    // which puts the 64 lanes of each write on distinct banks
    constexpr int ROW = HN + 4, COLS = GATED ? HN / 2 : HN, LANES = COLS / 8;
    static_assert(4 * 32 * ROW * 4 <= ring_bytes(BM, BN, false), "the epilogue uses the ring's LDS");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    float *w = reinterpret_cast<float *>(lds) + wave * 32 * ROW;
    constexpr int STEP = 64 / LANES, TURNS = 32 / STEP, TOGETHER = TURNS < 2 ? 1 : 2;
    const int r0 = lane / LANES, c = 8 * (lane % LANES), col = tn * FT + (wave & 1) * COLS + c, cols = p.N - col;
    const int first = tm * BM + (wave >> 1) * HM;
    const bool mine = cols > 0, whole = tn * FT + FT <= p.N;
    Columns<GATED> k;
    if (mine && p.splits <= 1)
        k.load(e, col, cols);
#pragma unroll 1
    for (int round = 0; round < FA / 2; ++round) {
        stage_rows(acc, round, w, ROW, lane);
        typedef float Rows[TOGETHER][8];
        auto rows = [&](auto take) {
#pragma unroll 1
            for (int q0 = 0; q0 < TURNS; q0 += TOGETHER) {
                const int lr = r0 + STEP * q0, row = first + 32 * round + lr;
                if (!mine || row >= p.M)
                    break;
                Rows v, u;
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
        if (p.splits > 1) {
            rows([&](int row, Rows &v, Rows &u) {
                const int ld = part_stride(p);
                float *to = p.part + part * part_size(p) + (size_t)row * ld + col;
#pragma unroll
                for (int q = 0; q < TOGETHER; ++q)
                    if (row + STEP * q < p.M) {
                        store8_f32(to + (size_t)(STEP * q) * ld, 8, v[q]);
                        if (GATED)
                            store8_f32(to + p.splits * part_size(p) + (size_t)(STEP * q) * ld, 8, u[q]);
                    }
            });
        } else {
            with_activation(e.act, [&](auto act) {
                rows([&](int row, Rows &v, Rows &u) {
                    if (whole)
                        emit_i8<GATED, true, decltype(act)::value, TOGETHER>(e, row, STEP, p.M, col, 8, v, u, k);
                    else
                        emit_i8<GATED, false, decltype(act)::value, TOGETHER>(e, row, STEP, p.M, col, cols, v, u, k);
                });
            });
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

template <int BM, int BN>
hipError_t launch_ring_as(const Product &p, const I8Epilogue &e, hipStream_t s)
{
    const dim3 grid((unsigned)(p.tiles_m * p.tiles_n), (unsigned)(p.splits > 1 ? p.splits : 1));
    if (p.gated)
        hipLaunchKernelGGL((i8_ring_kernel<BM, BN, true>), grid, dim3(256), 0, s, p, e);
    else
        hipLaunchKernelGGL((i8_ring_kernel<BM, BN, false>), grid, dim3(256), 0, s, p, e);
    return hipGetLastError();
}

// Adds the parts of a product whose sum was split, eight columns a thread.
template <bool GATED>
__global__ __launch_bounds__(256) void i8_join_kernel(Product p, I8Epilogue e)
{
    const int units = part_stride(p) / 8;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x, row = id / units;
    if (row >= p.M)
        return;
    const int col = 8 * (int)(id - row * units);
    Columns<GATED> k;
    k.load(e, col, p.N - col);
    auto sum = [&](const float *from, float (&f)[8]) {
        int t[8] = {};
        for (int s = 0; s < p.splits; ++s) {
            float v[8];
            load8_f32(from + s * part_size(p), 8, v);
#pragma unroll
            for (int c = 0; c < 8; ++c)
                t[c] += __float_as_int(v[c]);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c)
            f[c] = __int_as_float(t[c]);
    };
    const float *at = p.part + row * part_stride(p) + col;
    float v[1][8], u[1][8] = {};
    sum(at, v[0]);
    if (GATED)
        sum(at + p.splits * part_size(p), u[0]);
    with_activation(e.act, [&](auto act) {
        emit_i8<GATED, false, decltype(act)::value, 1>(e, (int)row, 0, p.M, col, p.N - col, v, u, k);
    });
}

// --------------------------------------------------------------- few rows --
//
// Bound by reading B once.  A workgroup of eight wavefronts takes a strip of 16
// columns (of each matrix) and the whole sum: wavefront w takes the 128-deep
// chunks w, w + 8, ... and has the loads of UNROLL of them in flight at once.  A
// load takes whole lines, eight rows x 128 bytes, and the wavefront passes the
// units through its own part of LDS into the lanes that multiply them: unit c of
// row r at 8 r + (c ^ ((r >> 1) & 7)).  The eight sums meet in LDS.
constexpr int kWaves = 8;

template <int RB, bool GATED, int UNROLL>
__global__ __launch_bounds__(64 * kWaves) void i8_rows_kernel(Product p, I8Epilogue e)
{
    constexpr int NB = GATED ? 2 : 1;
    constexpr int PITCH = 16 * NB + 4;                      // spreads four-row groups over the banks
    constexpr int SUMS = kWaves * RB * 16 * PITCH * 4, TURN = (RB + NB) * 2048;   // bytes; of a wavefront's chunk
    __shared__ __attribute__((aligned(1024))) uint8_t lds[SUMS > kWaves * TURN ? SUMS : kWaves * TURN];
    const int M = p.M, N = p.N, K = p.K;
    int none, strip;
    dgor_tile_of_block((int)blockIdx.x, 1, p.tiles_n, 1, none, strip);
    const int n0 = strip * kI8Strip;
    const int lane = threadIdx.x & 63, s16 = lane & 15, g = lane >> 4, r8 = lane >> 3, c8 = 8 * (lane & 7);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int chunks = (K + 63) / 64;   // of 64 pairs
    intx4 acc[RB][NB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b)
            acc[i][b] = intx4{0, 0, 0, 0};
    // rows past the matrices are read as the last: their sums are not used
    const uint16_t *rows_b[2 * NB], *rows_a[2 * RB];
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i)
        rows_b[i] = p.B.of(i / 2, 1) + (size_t)min(n0 + 8 * (i & 1) + r8, N - 1) * p.ldb;
#pragma unroll
    for (int i = 0; i < 2 * RB; ++i)
        rows_a[i] = p.A.of(0, 1) + (size_t)min(8 * i + r8, M - 1) * p.lda;
    u32x4 w[UNROLL][2 * NB], x[UNROLL][2 * RB];
    uint8_t *const xl = lds + wave * TURN, *const wl = xl + RB * 2048;
    auto slot = [&](int r) { return 16 * (8 * r + ((lane & 7) ^ ((r >> 1) & 7))); };
    for (int c0 = wave; c0 < chunks; c0 += kWaves * UNROLL) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int c = c0 + kWaves * u;
            if (c >= chunks)
                break;
            // K is whole units: one past it is A's zeros with any of B's
            const int k = 64 * c + c8, at = k < K ? k : 0;
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i)
                w[u][i] = *reinterpret_cast<const u32x4 *>(rows_b[i] + at);
#pragma unroll
            for (int i = 0; i < 2 * RB; ++i)
                x[u][i] = *reinterpret_cast<const u32x4 *>(rows_a[i] + at);
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int c = c0 + kWaves * u;
            if (c >= chunks)
                break;
            const bool inside = 64 * c + c8 < K;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i)
                *reinterpret_cast<u32x4 *>(wl + slot(8 * i + r8)) = w[u][i];
#pragma unroll
            for (int i = 0; i < 2 * RB; ++i)
                *reinterpret_cast<u32x4 *>(xl + slot(8 * i + r8)) = inside ? x[u][i] : u32x4{0u, 0u, 0u, 0u};
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                auto of_rows = [&](const uint8_t *at) {
                    return *reinterpret_cast<const intx4 *>(at + 16 * (8 * s16 + ((4 * h + g) ^ ((s16 >> 1) & 7))));
                };
                intx4 a[RB], b[NB];
#pragma unroll
                for (int i = 0; i < RB; ++i)
                    a[i] = of_rows(xl + 2048 * i);
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    b[j] = of_rows(wl + 2048 * j);
#pragma unroll
                for (int i = 0; i < RB; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[j], acc[i][j], 0, 0, 0);
            }
        }
    }
    __syncthreads();
    int *sums = reinterpret_cast<int *>(lds);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                sums[(wave * RB * 16 + 16 * i + 4 * g + r) * PITCH + 16 * b + s16] = acc[i][b][r];
    __syncthreads();
    for (int i = threadIdx.x; i < M * 16 * NB; i += 64 * kWaves) {
        int *q = sums + i / (16 * NB) * PITCH + i % (16 * NB);
        int v = q[0];
#pragma unroll
        for (int o = 1; o < kWaves; ++o)
            v += q[o * RB * 16 * PITCH];
        q[0] = v;
    }
    __syncthreads();
    for (int id = threadIdx.x; id < M * 2; id += 64 * kWaves) {
        const int row = id / 2, c = 8 * (id % 2), col = n0 + c;
        if (col >= N)
            continue;
        Columns<GATED> k;
        k.load(e, col, N - col);
        float v[1][8], u[1][8];
#pragma unroll
        for (int o = 0; o < 8; ++o) {
            v[0][o] = __int_as_float(sums[row * PITCH + c + o]);
            u[0][o] = GATED ? __int_as_float(sums[row * PITCH + 16 + c + o]) : 0.f;
        }
        with_activation(e.act, [&](auto act) {
            emit_i8<GATED, false, decltype(act)::value, 1>(e, row, 0, M, col, N - col, v, u, k);
        });
    }
}

template <int RB, bool GATED>
hipError_t launch_rows_as(const Product &p, const I8Epilogue &e, hipStream_t s)
{
    // 16-byte loads in flight, a lane: up to 32, what the registers hold
    constexpr int EACH = 2 * (RB + (GATED ? 2 : 1));
    constexpr int UNROLL = EACH <= 4 ? 8 : (EACH <= 8 ? 4 : 2);
    hipLaunchKernelGGL((i8_rows_kernel<RB, GATED, UNROLL>), dim3((unsigned)p.tiles_n), dim3(64 * kWaves), 0, s, p, e);
    return hipGetLastError();
}

template <bool GATED>
hipError_t launch_blocks(const Product &p, const I8Epilogue &e, hipStream_t s)
{
    switch ((p.M + 15) / 16) {
    case 1: return launch_rows_as<1, GATED>(p, e, s);
    case 2: return launch_rows_as<2, GATED>(p, e, s);
    case 3: return launch_rows_as<3, GATED>(p, e, s);
    case 4: return launch_rows_as<4, GATED>(p, e, s);
    default: return hipErrorInvalidValue;
    }
}

// ----------------------------------------------------------------- copies --
//
// A workgroup copies 4 KB: a unit of 16 bytes a thread, or a block of 64 x 64 that is
// transposed through LDS, where a thread turns four k of four columns round in
// registers.  Loads are at any address and none is in a branch: one that would
// leave the matrix takes the matrix's last bytes and is shifted.  (Blocks of 16 KB
// and bytes one by one at the edges: 8 us for 1000 x 777 and 777 x 1033.)

__device__ __forceinline__ void pack_rows(const I8Pack::Job &j, unsigned block)
{
    const long long units = j.ld_to / 16, id = (long long)block * 256 + threadIdx.x, row = id / units;
    if (row >= j.rows)
        return;
    const int c = 16 * (int)(id - row * units), n = j.cols - c;   // n bytes of the row, at least one
    const int8_t *from = j.from + row * j.ld;
    u32x4 v;
    if (j.cols >= 16) {
        v = *reinterpret_cast<const u32x4_at1 *>(from + min(c, j.cols - 16));
        if (n < 16) {
            const int s = 8 * (16 - n);
            uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
            lo = s < 64 ? lo >> s | hi << (64 - s) : hi >> (s - 64);
            hi = s < 64 ? hi >> s : 0;
            v = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
        }
    } else {
        uint32_t b[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
            b[e] = (uint8_t)from[min(e, n - 1)];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[e] |= 4 * e + i < n ? b[4 * e + i] << (8 * i) : 0u;
        }
    }
    *reinterpret_cast<u32x4 *>(j.to + row * j.ld_to + c) = v;
}

constexpr int kTurned = 64;   // a side of a transposed block

__device__ __forceinline__ void pack_turned(const I8Pack::Job &j, unsigned block, uint32_t *lds)
{
    typedef uint32_t u32_at1 __attribute__((aligned(1)));
    constexpr int PITCH = kTurned / 4 + 1;   // dwords of a column's k
    const int across = (j.rows + kTurned - 1) / kTurned;
    const int n0 = kTurned * (int)(block % across), k0 = kTurned * (int)(block / across);
    const int c = 4 * (int)(threadIdx.x & 15), k = 4 * (int)(threadIdx.x >> 4);   // of the block
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int kk = k0 + k + i, at = n0 + c;
        const int8_t *from = j.from + (long long)min(kk, j.cols - 1) * j.ld;
        if (j.rows >= 4) {
            const int first = min(at, j.rows - 4);
            const uint32_t v = *reinterpret_cast<const u32_at1 *>(from + first);
            r[i] = kk < j.cols && at - first < 4 ? v >> (8 * (at - first)) : 0u;
        } else {
            r[i] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t b = (uint8_t)from[min(at + e, j.rows - 1)];
                r[i] |= kk < j.cols && at + e < j.rows ? b << (8 * e) : 0u;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t v = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v |= ((r[i] >> (8 * e)) & 0xffu) << (8 * i);
        lds[(c + e) * PITCH + (threadIdx.x >> 4)] = v;
    }
    __syncthreads();
    const int n = (int)(threadIdx.x >> 2), u = (int)(threadIdx.x & 3);   // four units a column
    if (n0 + n < j.rows && k0 + 16 * u < j.ld_to) {
        const uint32_t *q = lds + n * PITCH + 4 * u;
        *reinterpret_cast<u32x4 *>(j.to + (long long)(n0 + n) * j.ld_to + k0 + 16 * u) = u32x4{q[0], q[1], q[2], q[3]};
    }
}

__global__ __launch_bounds__(256) void i8_pack_kernel(I8Pack r)
{
    __shared__ uint32_t lds[kTurned * (kTurned / 4 + 1)];
    const int i = r.jobs > 2 && blockIdx.x >= r.job[2].first ? 2 : (r.jobs > 1 && blockIdx.x >= r.job[1].first ? 1 : 0);
    const I8Pack::Job j = i == 2 ? r.job[2] : (i == 1 ? r.job[1] : r.job[0]);
    if (j.transpose)
        pack_turned(j, blockIdx.x - j.first, lds);
    else
        pack_rows(j, blockIdx.x - j.first);
}

}  // namespace

hipError_t launch_i8_ring(const Product &q, const I8Epilogue &e, RingTile tile, hipStream_t s)
{
    Product p = q;
    if (!p.trans_b || p.trans_a || p.nseg != 1 || p.nbatch != 1)
        return hipErrorInvalidValue;
    const int bm = ring_tile_m(tile), bn = ring_tile_n(tile), ft = p.gated ? bn / 2 : bn;
    p.tiles_m = (p.M + bm - 1) / bm;
    p.tiles_n = (p.N + ft - 1) / ft;
    p.group_m = 4;
    switch (tile) {
    case kRing256: return launch_ring_as<256, 256>(p, e, s);
    case kRing128: return launch_ring_as<128, 128>(p, e, s);
    case kRing128x64: return launch_ring_as<128, 64>(p, e, s);
    case kRing64: return launch_ring_as<64, 64>(p, e, s);
    default: return hipErrorInvalidValue;   // 256 x 128 is never the shortest on rows along k
    }
}

hipError_t launch_i8_rows(const Product &q, const I8Epilogue &e, hipStream_t s)
{
    Product p = q;
    if (!p.trans_b || p.trans_a || p.nseg != 1 || p.nbatch != 1 || p.M > kSkinnyRows || p.splits > 1)
        return hipErrorInvalidValue;
    p.tiles_m = 1;
    p.tiles_n = (p.N + kI8Strip - 1) / kI8Strip;
    return p.gated ? launch_blocks<true>(p, e, s) : launch_blocks<false>(p, e, s);
}

hipError_t launch_i8_join(const Product &p, const I8Epilogue &e, hipStream_t s)
{
    const long long threads = (long long)p.M * (part_stride(p) / 8);
    const dim3 grid((unsigned)((threads + 255) / 256));
    if (p.gated)
        hipLaunchKernelGGL((i8_join_kernel<true>), grid, dim3(256), 0, s, p, e);
    else
        hipLaunchKernelGGL((i8_join_kernel<false>), grid, dim3(256), 0, s, p, e);
    return hipGetLastError();
}

hipError_t launch_i8_pack(const I8Pack &q, hipStream_t s)
{
    I8Pack r = q;
    long long blocks = 0;
    for (int i = 0; i < r.jobs; ++i) {
        I8Pack::Job &j = r.job[i];
        j.first = (unsigned)blocks;
        blocks += j.transpose ? ((j.rows + kTurned - 1LL) / kTurned) * ((j.cols + kTurned - 1LL) / kTurned)
                              : ((long long)(j.ld_to / 16) * j.rows + 255) / 256;
    }
    if (blocks == 0)
        return hipSuccess;
    if (blocks >= (1 << 24))
        return hipErrorInvalidValue;
    hipLaunchKernelGGL(i8_pack_kernel, dim3((unsigned)blocks), dim3(256), 0, s, r);
    return hipGetLastError();
}

}  // namespace dgor
