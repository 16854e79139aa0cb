// Launches of the dense-layer, gated and layer-norm kernels, between the C
// entry points (linear.hip, norm.hip) and the kernel files.  Internal header.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "epilogue.h"

namespace dgor {

// One product Y = epilogue(op(A) op(B)) of 16-bit operands, op(A) M x K and
// op(B) K x N.  A is M x K (lda >= K) or, with trans_a, K x M; B is K x N or,
// with trans_b, N x K.
//   gated:  two products of one A, with both matrices of B; the epilogue gets
//           both sums of an element.
//   nseg:   the sum runs over that many pairs (segments) of an A and a B.
//   nbatch 2: two such products, of the pairs from 0 and from nseg, into e.Y
//           and Y1 in one launch.  (A gated one has one segment and batch.)
//   terms:  the pairs of each of up to two matrices.  An operand computed in FP32
//           is held as the sum of two bfloat16 terms, hi + lo, to 2^-17 of it:
//           two pairs, (hi, b) and (lo, b).  Three where the other operand is
//           binary16 and so two terms itself, exactly: hi hi, lo hi and hi lo (lo
//           lo is within the error).
// Split over k (splits > 1): split s covers stages [s chunk, (s + 1) chunk)
// of 64 k each (counted over all segments) and writes its FP32 sums to
// part: ((batch or gate/up) * splits + s) * part_size(p), rows padded to whole
// units; launch_join adds them in that order and applies the epilogue.
// One side's operands.  By distances and not as an array of pointers: an index
// into a kernel's argument that is not a constant puts a copy of the argument
// into scratch memory.
struct Side {
    const uint16_t *p;      // the first matrix
    long long matrix;       // bytes from it to the second
    long long term;         // bytes from a matrix to its lower term,
    int low;                // and which of a matrix's pairs takes that
    __host__ __device__ const uint16_t *of(int pair, int terms) const
    {
        const int second = pair >= terms, t = pair - (second ? terms : 0);
        return reinterpret_cast<const uint16_t *>(reinterpret_cast<const char *>(p) + (second ? matrix : 0) +
                                                  (t == low ? term : 0));
    }
};
struct Product {
    int M, N, K;
    Side A, B;
    int lda, ldb;
    bool bf16, trans_a, trans_b, gated;
    bool units;   // the operands' rows are whole 16-byte units, or padded to them
    bool opened;  // a binary16 operand has been opened into its terms (the few-row kernel opens it itself)
    int nseg, nbatch, terms;
    Epilogue e;
    void *Y1;
    int splits, chunk;
    float *part;
    int tiles_m, tiles_n, group_m;   // filled by the launcher
};

__host__ __device__ inline int part_stride(const Product &p) { return (p.N + 7) / 8 * 8; }
__host__ __device__ inline size_t part_size(const Product &p) { return (size_t)p.M * part_stride(p); }
constexpr int kStageDepth = 64;   // k per stage, the unit of Product::chunk
inline int product_stages(const Product &p) { return p.nseg * ((p.K + kStageDepth - 1) / kStageDepth); }
// The few-row kernel passes over each matrix B once, whatever its terms.
inline int row_stages(const Product &p) { return product_stages(p) / p.terms; }

// The register-staged tile (any operands).
constexpr int kTile = 64;
hipError_t launch_tile(const Product &p, hipStream_t stream);

// The rings: 16-byte aligned operands, rows of whole units of eight elements
// (or padded to them: the padding is read, zeros along k), strides below
// 2^22 and multiples of 8.
enum RingTile { kRing256, kRing256x128, kRing128, kRing128x64, kRing64 };
constexpr int ring_tile_m(RingTile t) { return t <= kRing256x128 ? 256 : (t == kRing64 ? 64 : 128); }
constexpr int ring_tile_n(RingTile t) { return t == kRing256 ? 256 : (t <= kRing128 ? 128 : 64); }
hipError_t launch_linear_ring(const Product &p, RingTile tile, hipStream_t stream);
// The two products of a backward pass (the weight's gradient, as K x M by K x N,
// and the input's) in one launch, on one of the three smaller tiles.
hipError_t launch_linear_ring_pair(const Product &weight, const Product &input, RingTile tile, hipStream_t stream);

// Few rows (at most kSkinnyRows, A as M x K, one product); each operand at
// least eight elements from its first to its last.  With terms A is bfloat16
// and in two terms, B whole and in the input format.
constexpr int kSkinnyRows = 64;
inline bool spans_a_unit(const Product &p)
{
    const long long b_rows = p.trans_b ? p.N : p.K, b_cols = p.trans_b ? p.K : p.N;
    return (long long)(p.M - 1) * p.lda + p.K >= 8 && (b_rows - 1) * p.ldb + b_cols >= 8;
}
// Columns of a workgroup's strip, of the one or each of the two products: what
// the registers hold of both products of a gated one, and of two terms of A.
inline int skinny_strip(const Product &p, bool split)
{
    const int rows = p.gated ? 32 : (p.terms > 1 ? 48 : kSkinnyRows);
    return p.trans_b ? 16 : (split && p.M <= rows ? 64 : 32);
}
hipError_t launch_linear_skinny(const Product &p, hipStream_t stream);

// Copies of operands whose rows are not whole units, padded to them with zeros;
// with `lo`, of a binary16 operand as two bfloat16 terms.
struct Repack {
    int jobs;
    struct Job {
        const uint16_t *from;
        uint16_t *to, *lo;
        int rows, cols, ld, ld_to;
        unsigned long long first;   // the job's first unit in the launch; filled by the launcher
    } job[3];
    unsigned long long units;       // of all jobs; filled by the launcher
    unsigned groups;                // workgroups that take them; filled by the launcher
};
hipError_t launch_repack(const Repack &r, hipStream_t stream);

hipError_t launch_join(const Product &p, hipStream_t stream);

// dZ = dY act'(Z) (Z null: dZ = dY, nothing written unless dz; rows padded
// with zeros to whole units) and each row block's column sums of the unrounded
// dZ, rounded to dbias where there is one block, else in FP32 to sums[block][N]
// (one of them, or neither).  Blocks of 64 rows, 16 where those would leave
// compute units idle.  dZ is rounded to the input format or, with dz_lo, held
// as two bfloat16 terms.  The copies `also` ride in the same launch.
inline int grad_rows(int M, int N) { return (M + 63LL) / 64 * ((N + 255) / 256) >= 1024 ? 64 : 16; }
constexpr int kGradCols = 256;   // of a workgroup
inline unsigned grad_groups(int M, int N)
{
    return (unsigned)((N + kGradCols - 1LL) / kGradCols) * (unsigned)((M + grad_rows(M, N) - 1LL) / grad_rows(M, N));
}
// Workgroups of launch_gate_grad, which take blocks of eight rows: four million
// at most, and as many turns as the blocks need.
inline unsigned gate_blocks(int M, int F) { return (unsigned)((F + kGradCols - 1LL) / kGradCols) * (unsigned)((M + 7LL) / 8); }
inline unsigned gate_groups(int M, int F) { return gate_blocks(M, F) < (1u << 22) ? gate_blocks(M, F) : 1u << 22; }
hipError_t launch_act_grad(int M, int N, const uint16_t *dy, int lddy, const uint16_t *z, int ldz, uint16_t *dz,
                           uint16_t *dz_lo, int lddz, int act, float *sums, uint16_t *dbias, const Repack &also, bool bf16,
                           hipStream_t stream);
// out[c] = sum over blocks of sums[block][c], in the input format.
hipError_t launch_sum_blocks(int blocks, int N, const float *sums, uint16_t *out, bool bf16, hipStream_t stream);
// dG = dH U act'(G), dU = dH act(G), held and padded likewise: [0] the value or
// its higher term, [1] null or the lower.
struct GateGrads {
    uint16_t *g[2], *u[2];
};
hipError_t launch_gate_grad(int M, int F, const uint16_t *dh, int lddh, const uint16_t *g, const uint16_t *u,
                            int ldp, const GateGrads &d, int ldd, int act, const Repack &also, bool bf16,
                            hipStream_t stream);

// Device check of the C entry points (api.hip): GEMM_OK on gfx950.
int device_status();

}  // namespace dgor
