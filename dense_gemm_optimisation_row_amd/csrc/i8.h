// Launches of the 8-bit products with scales, between the C entry points
// (linear_i8.hip) and the kernels (i8_kernels.hip).  Internal header.
#pragma once

#include "linear.h"

namespace dgor {

// What follows a product's INT32 sums: the scales of their row and column, bias,
// activation (or the gate's product) and residual, in FP32, and the rounding to
// the output's format.
struct I8Epilogue {
    const float *row, *col, *up;   // scales: M; N; N of the second matrix (gated)
    const float *bias;             // N, or null
    const void *R;                 // residual in the output's format, or null
    void *Y;
    int ldy, ldr, act, fmt;   // fmt: a Format
};

// The sum of a product of int8 operands overflows INT32 past this K: a code may
// be -128.
constexpr int kI8LongestK = 131071;

// The Product (linear.h) of int8 operands A, M x K, and B, N x K: K, lda and ldb
// count pairs of k, sixteen to a 32-byte row of 16-bit elements; A and B start on
// 16 bytes, K and the strides are multiples of 8 pairs.  trans_b, one segment, one
// batch.  Partial sums are INT32.
hipError_t launch_i8_ring(const Product &p, const I8Epilogue &e, RingTile tile, hipStream_t stream);
// At most kSkinnyRows rows.
constexpr int kI8Strip = 16;   // columns of a workgroup, of each matrix
hipError_t launch_i8_rows(const Product &p, const I8Epilogue &e, hipStream_t stream);
hipError_t launch_i8_join(const Product &p, const I8Epilogue &e, hipStream_t stream);

// Copies of operands as the products take them: rows of `cols` bytes at stride
// ld, or (transpose) cols rows of `rows` bytes, to `rows` rows at stride ld_to (a
// multiple of 16), padded with zeros.
struct I8Pack {
    int jobs;
    struct Job {
        const int8_t *from;
        int8_t *to;
        int rows, cols, ld, ld_to;
        bool transpose;
        unsigned first;   // the job's first workgroup; filled by the launcher
    } job[3];
};
hipError_t launch_i8_pack(const I8Pack &r, hipStream_t stream);

}  // namespace dgor
