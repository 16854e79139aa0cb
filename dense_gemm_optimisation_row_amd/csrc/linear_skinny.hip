// The dense-layer products of few rows (a decoding step): Y = epilogue(A op(B))
// for M of at most 64.
//
// Bound by reading B once.  A workgroup of eight wavefronts takes a strip of
// 16 (or 32) columns and the whole sum over k, so there is one launch and
// nothing to join: wavefront w takes the 64-deep chunks w, w + 8, ... and has
// the loads of UNROLL of them in flight at once; the eight sums meet in LDS,
// in wavefront order.  Operands go from memory to registers; A, which every
// workgroup reads, comes from the caches.  FP32 sums on v_mfma_f32_16x16x32:
// lane (g, s) = (lane / 16, lane % 16) supplies k 8 g .. 8 g + 7 of row s of A
// and of column s of B.  B as N x K has those eight k together: one 16-byte
// load.  Of B as K x N a lane loads eight columns of one k row, and the
// wavefront passes 32 rows x 16 columns through 1 KB of LDS to transposing
// reads; row positions 4 g + j and 16 + 4 g + j hold k 8 g + j and 8 g + 4 + j,
// so that each read is of contiguous bytes.  A strip's 32-byte row pieces of
// a K x N matrix are parts of lines that the strips beside it want too: these
// run on the same XCD, which fetches each line once.
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
    static __device__ __forceinline__ floatx4 mfma(u32x4 a, u32x4 b, floatx4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(halfx8, a), __builtin_bit_cast(halfx8, b), c,
                                                      0, 0, 0);
    }
};
struct OpBrain : Brain16 {
    static __device__ __forceinline__ floatx4 mfma(u32x4 a, u32x4 b, floatx4 c)
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

constexpr int kWaves = 8;

// RB: 16-row blocks of A; CB: 16-column blocks of a strip.  A gated product's
// blocks are CB of the gate and then the same CB of the up projection.
template <class Op, int RB, int CB, bool TB, bool GATED, int UNROLL>
__global__ __launch_bounds__(64 * kWaves) void linear_skinny_kernel(Product p)
{
    constexpr int NB = GATED ? 2 * CB : CB;
    constexpr int PITCH = 16 * NB + 4;                      // floats; spreads four-row groups over the banks
    constexpr int SUMS = kWaves * RB * 16 * PITCH * 4;      // bytes
    constexpr int TURN = TB ? 0 : kWaves * 2 * NB * 1024;
    __shared__ __attribute__((aligned(16))) uint8_t lds[SUMS > TURN ? SUMS : TURN];
    const int M = p.M, N = p.N, K = p.K;
    int none, strip;
    dgor_tile_of_block((int)blockIdx.x, 1, p.tiles_n, 1, none, strip);
    const int n0 = strip * 16 * CB;
    const int lane = threadIdx.x & 63, s16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int per_seg = (K + 63) / 64, chunks = p.nseg * per_seg;
    const int pos = lane >> 1;                              // row position of this lane's piece of B as K x N
    const int krow = pos < 16 ? 8 * (pos >> 2) + (pos & 3) : 8 * ((pos - 16) >> 2) + 4 + (pos & 3);

    u32x4 w[UNROLL][2][NB], x[UNROLL][2][RB];
    auto fetch = [&](int c0, bool whole) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int c = c0 + kWaves * u, seg = c >= per_seg ? p.nseg - 1 : 0;
            const int k0 = 64 * (c - seg * per_seg);
            const uint16_t *A = p.A[seg];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = k0 + 32 * h;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint16_t *B = p.B[GATED ? b / CB : seg];
                    const int n = n0 + 16 * (b % CB);
                    if (TB) {
                        w[u][h][b] = whole ? load8_16(B + (size_t)(n + s16) * p.ldb + k + 8 * g, 8)
                                           : load_unit(B, p.ldb, n + s16, N, k + 8 * g, K);
                    } else {
                        const int col = n + 8 * (lane & 1);
                        w[u][h][b] = whole ? load8_16(B + (size_t)(k + krow) * p.ldb + col, 8)
                                           : load_unit(B, p.ldb, k + krow, K, col, N);
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < RB; ++i)
                    x[u][h][i] = load_unit(A, p.lda, 16 * i + s16, M, k0 + 32 * h + 8 * g,
                                           whole ? 0x7fffffff : K);
        }
    };
    floatx4 acc[RB][NB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b)
            acc[i][b] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int c0 = wave; c0 < chunks; c0 += kWaves * UNROLL) {
        const int last = c0 + kWaves * (UNROLL - 1);
        const bool full_k = p.nseg == 1 ? 64 * (last + 1) <= K : K % 64 == 0 && last < chunks;
        if (full_k && n0 + 16 * CB <= N)
            fetch(c0, true);
        else
            fetch(c0, false);
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (!TB) {
                uint8_t *mine = lds + wave * 2 * NB * 1024;
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        *reinterpret_cast<u32x4 *>(mine + (h * NB + b) * 1024 + 16 * lane) = w[u][h][b];
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const uint8_t *q = mine + (h * NB + b) * 1024 + 8 * lane;
                        const shortx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4 *)q);
                        const shortx4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4 *)(q + 512));
                        w[u][h][b] =
                            __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                    }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < RB; ++i)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        acc[i][b] = Op::mfma(x[u][h][i], w[u][h][b], acc[i][b]);
        }
    }

    // the wavefronts' sums, added in their order
    if (!TB)
        __syncthreads();
    float *sums = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                sums[(wave * RB * 16 + 16 * i + 4 * g + r) * PITCH + 16 * b + s16] = acc[i][b][r];
    __syncthreads();
    for (int e = threadIdx.x; e < M * 16 * NB; e += 64 * kWaves) {
        float *q = sums + e / (16 * NB) * PITCH + e % (16 * NB);
        float v = q[0];
#pragma unroll
        for (int o = 1; o < kWaves; ++o)
            v += q[o * RB * 16 * PITCH];
        q[0] = v;
    }
    __syncthreads();
    for (int id = threadIdx.x; id < M * 2 * CB; id += 64 * kWaves) {
        const int row = id / (2 * CB), c = 8 * (id % (2 * CB)), col = n0 + c;
        if (col < N) {
            float v[8], u[8];
#pragma unroll
            for (int o = 0; o < 8; ++o) {
                v[o] = sums[row * PITCH + c + o];
                u[o] = GATED ? sums[row * PITCH + 16 * CB + c + o] : 0.f;
            }
            emit8<Op, GATED>(p.e, row, col, N - col, v, u);
        }
    }
}

template <class Op, int RB, int CB, bool TB, bool GATED>
hipError_t launch_rows(const Product &p, hipStream_t s)
{
    // loads in flight: 16 of B and as many of A for one row block, what the
    // registers hold beyond it
    constexpr int UNROLL = RB == 1 && CB == 1 && !GATED ? 8 : 4;
    hipLaunchKernelGGL((linear_skinny_kernel<Op, RB, CB, TB, GATED, UNROLL>), dim3((unsigned)p.tiles_n),
                       dim3(64 * kWaves), 0, s, p);
    return hipGetLastError();
}

template <class Op, int CB, bool TB, bool GATED>
hipError_t launch_blocks(const Product &p, hipStream_t s)
{
    switch ((p.M + 15) / 16) {
    case 1: return launch_rows<Op, 1, CB, TB, GATED>(p, s);
    case 2: return launch_rows<Op, 2, CB, TB, GATED>(p, s);
    case 3: return launch_rows<Op, 3, CB, TB, GATED>(p, s);
    case 4: return launch_rows<Op, 4, CB, TB, GATED>(p, s);
    default: return hipErrorInvalidValue;
    }
}

template <class Op>
hipError_t launch_op(const Product &p, int strip, hipStream_t s)
{
    if (p.gated)
        return p.trans_b ? launch_blocks<Op, 1, true, true>(p, s) : launch_blocks<Op, 1, false, true>(p, s);
    if (strip == 32)
        return p.trans_b ? launch_blocks<Op, 2, true, false>(p, s) : launch_blocks<Op, 2, false, false>(p, s);
    return p.trans_b ? launch_blocks<Op, 1, true, false>(p, s) : launch_blocks<Op, 1, false, false>(p, s);
}

}  // namespace

hipError_t launch_linear_skinny(const Product &q, int strip, hipStream_t s)
{
    Product p = q;
    if (p.trans_a || p.nbatch != 1 || p.M > kSkinnyRows || (strip != 16 && (strip != 32 || p.gated)))
        return hipErrorInvalidValue;
    p.tiles_m = 1;
    p.tiles_n = (p.N + strip - 1) / strip;
    return p.bf16 ? launch_op<OpBrain>(p, strip, s) : launch_op<OpHalf>(p, strip, s);
}

}  // namespace dgor
