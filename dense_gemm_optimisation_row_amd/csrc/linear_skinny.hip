// The dense-layer products of few rows (a decoding step): Y = epilogue(A op(B))
// for M of at most 64.
//
// Bound by reading B once.  A workgroup of eight wavefronts takes a strip of
// columns and, as a rule, the whole sum over k, so there is one launch and
// nothing to join: wavefront w takes the 64-deep chunks w, w + 8, ... and has the
// loads of UNROLL of them in flight at once; the eight sums meet in LDS, in
// wavefront order.  FP32 sums on v_mfma_f32_16x16x32: lane (g, s) = (lane / 16,
// lane % 16) supplies k 8 g .. 8 g + 7 of row s of A and of column s of B.
//
// What the caches serve is counted in pieces that neighbouring lanes ask for
// together, so every load takes whole rows of a chunk (of A, and of B as
// N x K: 8 rows x 128 bytes; of B as K x N: 16 rows x the strip's 64 bytes)
// and the wavefront passes the units through its own part of LDS into the
// lanes that multiply them.  Loaded in the multiplying lanes' order, 16 bytes
// from each of 16 rows, a 48 x 4096 by 4096 x 4096 product took 18.6 us.
//   16 rows x 64 k (2 KB): unit c of row r at 8 r + (c ^ ((r >> 1) & 7)), read
//     128 bits a lane;
//   64 k x 32 columns (4 KB, in 16-row loads j): the load's rows 4 q + i hold
//     k 32 (j / 2) + 4 (j % 2) + 8 q + i, unit u of row r at 4 r + (u ^ 2 ((r >> 2) & 1)),
//     read transposing, the eight rows of a cycle on distinct banks.
//   64 k x 64 columns (8 KB): unit u of row k at 8 k + (u ^ x(k)).
// Strips: 16 columns of B as N x K, 32 as K x N; the strips beside it, which
// share its lines, run on the same XCD.  A compute unit takes about the same
// number of pieces a microsecond whatever their size (K x N: 32 bytes each 19
// GB/s, 64 bytes 33), so of a K x N matrix with a long sum the strips are 64
// columns, whole lines, and the sum is split over workgroups and joined.
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

// A binary16 matrix B with A in bfloat16 terms: B's fragments are opened into
// two terms (exactly) where they are multiplied.
struct OpOpened : Half16 {
    static __device__ __forceinline__ floatx4 mfma(u32x4 a, u32x4 b, floatx4 c) { return OpBrain::mfma(a, b, c); }
};

constexpr int kWaves = 8;

// Of 64 k rows of eight units: unit u of row k at 8 k + (u ^ this); k and k + 4
// have the same.
__device__ __forceinline__ int wide_swizzle(int k) { return 2 * ((k >> 1) & 1) + 4 * ((k >> 3) & 1); }

// RB: 16-row blocks of A; CB: 16-column blocks of a strip.  A gated product's
// blocks are CB of the gate and then the same CB of the up projection.  TERMS:
// as Product's; B is read once, A's two terms pass through the same LDS one
// after the other.
template <class Op, int RB, int CB, bool TB, bool GATED, int TERMS, int UNROLL>
__global__ __launch_bounds__(64 * kWaves) void linear_skinny_kernel(Product p)
{
    constexpr int NM = GATED ? 2 : 1, NB = NM * CB;         // matrices B, column blocks
    constexpr int AT = TERMS > 1 ? 2 : 1;                   // terms of A
    static_assert(TB || CB == 2 || CB == 4, "a K x N strip is 32 or 64 columns");
    static_assert(!GATED || TERMS == 1, "a gated product's A is in the input format");
    constexpr int PITCH = 16 * NB + 4;                      // floats; spreads four-row groups over the banks
    constexpr int SUMS = kWaves * RB * 16 * PITCH * 4;      // bytes
    constexpr int TURN = (RB + NB) * 2048;                  // a wavefront's chunk
    __shared__ __attribute__((aligned(1024))) uint8_t lds[SUMS > kWaves * TURN ? SUMS : kWaves * TURN];
    const int M = p.M, N = p.N, K = p.K;
    int none, strip;
    dgor_tile_of_block((int)blockIdx.x, 1, p.tiles_n, 1, none, strip);
    const int n0 = strip * 16 * CB;
    const int lane = threadIdx.x & 63, s16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int per_seg = (K + 63) / 64;
    const int first = p.splits > 1 ? (int)blockIdx.y * p.chunk : 0;
    const int segs = p.nseg / TERMS;                        // matrices B of the sum
    const int chunks = p.splits > 1 ? min(first + p.chunk, segs * per_seg) : segs * per_seg;
    const int r8 = lane >> 3, c8 = 8 * (lane & 7);          // of 8 rows x 64 k
    const int r16 = lane >> 2, c4 = 8 * (lane & 3);         // of 16 rows x 32 columns

    u32x4 w[UNROLL][2 * NB], x[UNROLL][AT][2 * RB];
    // where chunk c begins, and its operands
    struct Chunk {
        int k0;
        Operand a[AT], b[NM];
    };
    auto chunk_of = [&](int c) {
        const int seg = c >= per_seg ? segs - 1 : 0;   // of one or two
        Chunk s;
        s.k0 = 64 * (c - seg * per_seg);
#pragma unroll
        for (int t = 0; t < AT; ++t)
            s.a[t] = Operand{p.A.of(seg * TERMS + t, TERMS), M, K, (size_t)p.lda};
#pragma unroll
        for (int i = 0; i < NM; ++i)
            s.b[i] = Operand{p.B.of(GATED ? i : seg * TERMS, TERMS), TB ? N : K, TB ? K : N, (size_t)p.ldb};
        return s;
    };
    // load i of B: the (i % 2 CB)th of matrix i / (2 CB)
    auto b_place = [&](int i, int k0, int &row, int &col) {
        const int j = i % (2 * CB);
        if (TB)
            row = n0 + 8 * j + r8, col = k0 + c8;
        else if (CB == 4)
            row = k0 + 8 * j + r8, col = n0 + c8;
        else
            row = k0 + 32 * (j >> 1) + 4 * (j & 1) + 8 * (r16 >> 2) + (r16 & 3), col = n0 + c4;
    };
    floatx4 acc[RB][NB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b)
            acc[i][b] = floatx4{0.f, 0.f, 0.f, 0.f};
    uint8_t *const xl = lds + wave * TURN, *const wl = xl + RB * 2048;
    auto row_slot = [&](int r) { return 16 * (8 * r + ((lane & 7) ^ ((r >> 1) & 7))); };
    for (int c0 = first + wave; c0 < chunks; c0 += kWaves * UNROLL) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const Chunk s = chunk_of(c0 + kWaves * u);
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) {
                int row, col;
                b_place(i, s.k0, row, col);
                w[u][i] = s.b[i / (2 * CB)].load(row, col);
            }
#pragma unroll
            for (int t = 0; t < AT; ++t)
#pragma unroll
                for (int i = 0; i < 2 * RB; ++i) {
                    x[u][t][i] = u32x4{0u, 0u, 0u, 0u};
                    if (8 * i + r8 < M)
                        x[u][t][i] = s.a[t].load(8 * i + r8, s.k0 + c8);
                }
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int c = c0 + kWaves * u;
            if (c >= chunks)
                break;
            const Chunk s = chunk_of(c);
            if (s.k0 + 64 > K || n0 + 16 * CB > N) {
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) {
                    int row, col;
                    b_place(i, s.k0, row, col);
                    w[u][i] = s.b[0].settle(w[u][i], row, col);
                }
#pragma unroll
                for (int t = 0; t < AT; ++t)
#pragma unroll
                    for (int i = 0; i < 2 * RB; ++i)
                        x[u][t][i] = s.a[t].settle(x[u][t][i], 8 * i + r8, s.k0 + c8);
            }
#pragma unroll
            for (int t = 0; t < AT; ++t) {
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                if (t == 0)
#pragma unroll
                    for (int i = 0; i < 2 * NB; ++i)
                        *reinterpret_cast<u32x4 *>(
                            wl +
                            (TB ? row_slot(8 * i + r8)
                                : 1024 * i + (CB == 4 ? 128 * r8 + 16 * ((lane & 7) ^ wide_swizzle(8 * i + r8))
                                                      : 64 * r16 + 16 * ((lane & 3) ^ (2 * ((r16 >> 2) & 1)))))) = w[u][i];
#pragma unroll
                for (int i = 0; i < 2 * RB; ++i)
                    *reinterpret_cast<u32x4 *>(xl + row_slot(8 * i + r8)) = x[u][t][i];
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    auto of_rows = [&](const uint8_t *at) {
                        return *reinterpret_cast<const u32x4 *>(at + 16 * (8 * s16 + ((4 * h + g) ^ ((s16 >> 1) & 7))));
                    };
                    u32x4 a[RB], b[NB];
#pragma unroll
                    for (int i = 0; i < RB; ++i)
                        a[i] = of_rows(xl + 2048 * i);
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        if (TB) {
                            b[j] = of_rows(wl + 2048 * j);
                        } else {
                            const int unit = 2 * (j % CB) + ((s16 & 3) >> 1), kr = 8 * g + (s16 >> 2);
                            const uint8_t *q = wl + 2048 * CB * (j / CB) + 1024 * CB * h + 8 * (s16 & 1) +
                                               (CB == 4 ? 128 * kr + 16 * (unit ^ wide_swizzle(kr))
                                                        : 64 * (4 * g + (s16 >> 2)) + 16 * (unit ^ (2 * (g & 1))));
                            const shortx4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4 *)q);
                            const shortx4 hi =
                                __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4 *)(q + (CB == 4 ? 512 : 1024)));
                            b[j] = __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                        }
                    }
                    u32x4 low[NB];
                    if (TERMS == 3)
#pragma unroll
                        for (int j = 0; j < NB; ++j) {
                            float f[8];
                            unpack8<Half16>(b[j], f);
                            pack8_terms(f, b[j], low[j]);
                        }
#pragma unroll
                    for (int i = 0; i < RB; ++i)
#pragma unroll
                        for (int j = 0; j < NB; ++j) {
                            acc[i][j] = Op::mfma(a[i], b[j], acc[i][j]);
                            if (TERMS == 3 && t == 0)
                                acc[i][j] = Op::mfma(a[i], low[j], acc[i][j]);
                        }
                }
            }
        }
    }

    // the wavefronts' sums, added in their order
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
            if (p.splits > 1) {
                float *part = p.part + blockIdx.y * part_size(p) + (size_t)row * part_stride(p) + col;
                store8_f32(part, 8, v);
                if (GATED)
                    store8_f32(part + p.splits * part_size(p), 8, u);
            } else {
                emit8<Op, GATED>(p.e, row, col, N - col, v, u);
            }
        }
    }
}

template <class Op, int RB, int CB, bool TB, bool GATED, int TERMS>
hipError_t launch_rows(const Product &p, hipStream_t s)
{
    // 16-byte loads in flight, a lane: up to 32, what the registers hold
    constexpr int EACH = 2 * ((TERMS > 1 ? 2 : 1) * RB + CB * (GATED ? 2 : 1));
    constexpr int UNROLL = EACH <= 4 ? 8 : (EACH <= 8 ? 4 : (EACH <= 12 ? 2 : 1));
    hipLaunchKernelGGL((linear_skinny_kernel<Op, RB, CB, TB, GATED, TERMS, UNROLL>),
                       dim3((unsigned)p.tiles_n, (unsigned)(p.splits > 1 ? p.splits : 1)), dim3(64 * kWaves), 0, s, p);
    return hipGetLastError();
}

template <class Op, int CB, bool TB, bool GATED, int TERMS = 1>
hipError_t launch_blocks(const Product &p, hipStream_t s)
{
    switch ((p.M + 15) / 16) {
    case 1: return launch_rows<Op, 1, CB, TB, GATED, TERMS>(p, s);
    case 2: return launch_rows<Op, 2, CB, TB, GATED, TERMS>(p, s);
    case 3: return launch_rows<Op, 3, CB, TB, GATED, TERMS>(p, s);
    case 4: return launch_rows<Op, 4, CB, TB, GATED, TERMS>(p, s);
    default: return hipErrorInvalidValue;
    }
}

template <class Op, int TERMS>
hipError_t launch_plain(const Product &p, int strip, hipStream_t s)
{
    if (p.trans_b)
        return launch_blocks<Op, 1, true, false, TERMS>(p, s);
    if (strip == 32)
        return launch_blocks<Op, 2, false, false, TERMS>(p, s);
    if constexpr (TERMS > 1)
        switch ((p.M + 15) / 16) {
        case 1: return launch_rows<Op, 1, 4, false, false, TERMS>(p, s);
        case 2: return launch_rows<Op, 2, 4, false, false, TERMS>(p, s);
        default: return launch_rows<Op, 3, 4, false, false, TERMS>(p, s);
        }
    else
        return launch_blocks<Op, 4, false, false>(p, s);
}

template <class Op>
hipError_t launch_op(const Product &p, int strip, hipStream_t s)
{
    if (!p.gated)
        return launch_plain<Op, 1>(p, strip, s);
    if (p.trans_b)
        return launch_blocks<Op, 1, true, true>(p, s);
    if (strip == 32)
        return launch_blocks<Op, 2, false, true>(p, s);
    return p.M <= 16 ? launch_rows<Op, 1, 4, false, true, 1>(p, s) : launch_rows<Op, 2, 4, false, true, 1>(p, s);
}

}  // namespace

hipError_t launch_linear_skinny(const Product &q, hipStream_t s)
{
    Product p = q;
    if (p.trans_a || p.nbatch != 1 || p.M > kSkinnyRows || !spans_a_unit(p) || p.opened || p.nseg > 2 * p.terms)
        return hipErrorInvalidValue;
    const int strip = skinny_strip(p, p.splits > 1);
    p.tiles_m = 1;
    p.tiles_n = (p.N + strip - 1) / strip;
    if (p.terms == 3)
        return launch_plain<OpOpened, 3>(p, strip, s);
    if (p.terms == 2)
        return launch_plain<OpBrain, 2>(p, strip, s);
    return p.bf16 ? launch_op<OpBrain>(p, strip, s) : launch_op<OpHalf>(p, strip, s);
}

}  // namespace dgor
