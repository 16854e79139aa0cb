// The element-wise work around the dense layers' products: copies of operands
// whose rows are not whole 16-byte units, and of the backward passes the gradient
// of the pre-activations and the bias gradient's column sums of the unrounded
// values.
//
// The gradient is computed in FP32 and the matrix cores take 16 bits.  It is
// written as the sum of two bfloat16 terms, so that each product of it is within
// 2^-17 of that of the FP32 values and has their range: rounded once to
// bfloat16 it would add as much error to dX and dW as their own rounding does
// (1.66e-3 in all, 2.35e-3 so), and in binary16 it would overflow past 65504 and
// vanish below 2^-25.  The caller may ask for the rounding, which halves (binary16:
// takes a third of) the products' work.
//
// Bound by memory: each value is read once and written once, or as two terms.  A
// workgroup covers 64 (or 16) rows x 256 columns, 32 lanes of eight columns times 8
// rows at a time, so a row's accesses are 512 contiguous bytes and the column sums
// of a workgroup need one pass through LDS.  The sums go out per row block and are
// added in block order by a second kernel, so they do not depend on which
// workgroup finished first.
#include "linear.h"

namespace dgor {
namespace {

constexpr int kCols = kGradCols;

// Workgroup `group` of a copy: a unit a thread (further units where there are
// more than the workgroups take at once), read at any alignment, written whole.
__device__ __forceinline__ void repack(const Repack &r, unsigned group)
{
    for (unsigned long long id = group * 256ULL + threadIdx.x; id < r.units; id += r.groups * 256ULL) {
        Repack::Job j = r.job[0];
#pragma unroll
        for (int i = 1; i < 3; ++i)
            if (i < r.jobs && id >= r.job[i].first)
                j = r.job[i];
        // a job has fewer than 2^32 units: 2^22 blocks of 128 x 64 elements at most
        const unsigned per = (unsigned)(j.cols + 7) / 8, u = (unsigned)(id - j.first), row = u / per;
        const int col = 8 * (int)(u - row * per);
        u32x4 v = load8_16(j.from + (size_t)row * j.ld + col, j.cols - col);
        const size_t at = (size_t)row * j.ld_to + col;
        if (j.lo) {
            float f[8];
            u32x4 lo;
            unpack8<Half16>(v, f);
            pack8_terms(f, v, lo);
            store8_16(j.lo + at, 8, lo);
        }
        store8_16(j.to + at, 8, v);
    }
}

// d in the input format or, where there is a lower term, as two.
template <class Fmt>
__device__ __forceinline__ void store_gradient(uint16_t *hi, uint16_t *lo, size_t at, const float (&d)[8])
{
    u32x4 v, w;
    if (lo) {
        pack8_terms(d, v, w);
        store8_16(lo + at, 8, w);
    } else {
        v = pack8<Fmt>(d);
    }
    store8_16(hi + at, 8, v);
}

// x to act'(x): one uniform branch on the activation, not one an element.
__device__ __forceinline__ void slopes(int act, float (&x)[8])
{
    auto apply = [&](int a) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float value;
            activate_slope(a, x[e], value, x[e]);
        }
    };
    switch (act) {
    case GEMM_ACT_RELU: apply(GEMM_ACT_RELU); break;
    case GEMM_ACT_GELU: apply(GEMM_ACT_GELU); break;
    case GEMM_ACT_GELU_TANH: apply(GEMM_ACT_GELU_TANH); break;
    case GEMM_ACT_SILU: apply(GEMM_ACT_SILU); break;
    default: apply(GEMM_ACT_NONE);
    }
}

// R: rows of a thread.
template <class Fmt, int R>
__global__ __launch_bounds__(256) void act_grad_kernel(int M, int N, const uint16_t *__restrict__ dy, int lddy,
                                                       const uint16_t *__restrict__ z, int ldz,
                                                       uint16_t *__restrict__ dz, uint16_t *__restrict__ dz_lo,
                                                       int lddz, int act, float *__restrict__ sums, uint16_t *__restrict__ dbias,
                                                       Repack also, unsigned groups)
{
    if (blockIdx.x >= groups) {
        repack(also, blockIdx.x - groups);
        return;
    }
    __shared__ float part[8][kCols + 8];
    const int lane = threadIdx.x & 31, r8 = threadIdx.x >> 5;
    const int strips = (N + kCols - 1) / kCols, strip = blockIdx.x % strips, block = blockIdx.x / strips;
    const int col = strip * kCols + 8 * lane, n = N - col;
    const int row0 = block * 8 * R;
    float total[8] = {};
    // all of a thread's rows are loaded before the first is worked on; rows
    // past M are read from the last and not used
    auto rows = [&](auto load) {
        u32x4 dv[R], zv[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const size_t row = (size_t)min(row0 + 8 * i + r8, M - 1);
            dv[i] = load(dy + row * lddy + col);
            if (z)
                zv[i] = load(z + row * ldz + col);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = row0 + 8 * i + r8;
            if (row >= M)
                break;
            float d[8];
            unpack8<Fmt>(dv[i], d);
            if (z) {
                float x[8];
                unpack8<Fmt>(zv[i], x);
                slopes(act, x);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    d[e] *= x[e];
            }
            if (dz)   // past N zeros: its rows are padded to whole units
                store_gradient<Fmt>(dz, dz_lo, (size_t)row * lddz + col, d);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                total[e] += d[e];
        }
    };
    if (n >= 8)
        rows([](const uint16_t *p) { return load8_16(p, 8); });
    else if (n > 0)
        rows([&](const uint16_t *p) { return load8_16(p, n); });
    if (!sums && !dbias)
        return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        part[r8][8 * lane + e] = total[e];
    __syncthreads();
    const int c = strip * kCols + threadIdx.x;
    if (c < N) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r)
            s += part[r][threadIdx.x];
        if (sums)
            sums[(size_t)block * N + c] = s;
        else
            dbias[c] = Fmt::down(s);
    }
}

template <class Fmt>
__global__ __launch_bounds__(256) void sum_blocks_kernel(int blocks, int N, const float *__restrict__ sums,
                                                         uint16_t *__restrict__ out)
{
    // 32 columns x 8 threads over the blocks
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < N)
#pragma unroll 4
        for (int b = w; b < blocks; b += 8)
            s += sums[(size_t)b * N + c];
    part[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < N)
        out[c] = Fmt::down(((part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane])) +
                           ((part[4][lane] + part[5][lane]) + (part[6][lane] + part[7][lane])));
}

template <class Fmt>
__global__ __launch_bounds__(256) void gate_grad_kernel(int M, int F, const uint16_t *__restrict__ dh, int lddh,
                                                        const uint16_t *__restrict__ g,
                                                        const uint16_t *__restrict__ u, int ldp,
                                                        GateGrads out, int ldd, int act, Repack also,
                                                        unsigned groups, unsigned blocks)
{
    if (blockIdx.x >= groups) {
        repack(also, blockIdx.x - groups);
        return;
    }
    // a unit a thread, 32 units x 8 rows a workgroup
    const int lane = threadIdx.x & 31, r8 = threadIdx.x >> 5;
    const unsigned strips = (unsigned)(F + kCols - 1) / kCols;
    for (unsigned block = blockIdx.x; block < blocks; block += groups) {
        const int col = (int)(block % strips) * kCols + 8 * lane, n = F - col;
        const int row = (int)(block / strips) * 8 + r8;
        if (n <= 0 || row >= M)
            continue;
        u32x4 dv, gv, uv;
        const size_t at = (size_t)row * ldp + col;
        if (n >= 8) {
            dv = load8_16(dh + (size_t)row * lddh + col, 8);
            gv = load8_16(g + at, 8);
            uv = load8_16(u + at, 8);
        } else {
            dv = load8_16(dh + (size_t)row * lddh + col, n);
            gv = load8_16(g + at, n);
            uv = load8_16(u + at, n);
        }
        float d[8], x[8], y[8], a[8], b[8];
        unpack8<Fmt>(dv, d);
        unpack8<Fmt>(gv, x);
        unpack8<Fmt>(uv, y);
        auto apply = [&](int which) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float value, slope;
                activate_slope(which, x[e], value, slope);
                a[e] = d[e] * y[e] * slope;
                b[e] = d[e] * value;
            }
        };
        switch (act) {
        case GEMM_ACT_RELU: apply(GEMM_ACT_RELU); break;
        case GEMM_ACT_GELU: apply(GEMM_ACT_GELU); break;
        case GEMM_ACT_GELU_TANH: apply(GEMM_ACT_GELU_TANH); break;
        case GEMM_ACT_SILU: apply(GEMM_ACT_SILU); break;
        default: apply(GEMM_ACT_NONE);
        }
        store_gradient<Fmt>(out.g[0], out.g[1], (size_t)row * ldd + col, a);   // past F zeros
        store_gradient<Fmt>(out.u[0], out.u[1], (size_t)row * ldd + col, b);
    }
}

__global__ __launch_bounds__(256) void repack_kernel(Repack r) { repack(r, blockIdx.x); }

// Counts the jobs' units; returns the workgroups that take them, a million at
// most.
unsigned repack_groups(Repack &r)
{
    r.units = 0;
    for (int i = 0; i < r.jobs; ++i) {
        r.job[i].first = r.units;
        r.units += (unsigned long long)r.job[i].rows * ((r.job[i].cols + 7LL) / 8);
    }
    const unsigned long long groups = (r.units + 255) / 256;
    return r.groups = (unsigned)(groups < (1 << 20) ? groups : (1 << 20));
}

}  // namespace

hipError_t launch_repack(const Repack &q, hipStream_t s)
{
    Repack r = q;
    const unsigned groups = repack_groups(r);
    if (groups)
        hipLaunchKernelGGL(repack_kernel, dim3(groups), dim3(256), 0, s, r);
    return hipGetLastError();
}

hipError_t launch_act_grad(int M, int N, const uint16_t *dy, int lddy, const uint16_t *z, int ldz, uint16_t *dz,
                           uint16_t *dz_lo, int lddz, int act, float *sums, uint16_t *dbias, const Repack &q, bool bf16,
                           hipStream_t s)
{
    Repack also = q;
    const unsigned groups = grad_groups(M, N);
    const auto kernel = grad_rows(M, N) == 64 ? (bf16 ? act_grad_kernel<Brain16, 8> : act_grad_kernel<Half16, 8>)
                                   : (bf16 ? act_grad_kernel<Brain16, 2> : act_grad_kernel<Half16, 2>);
    hipLaunchKernelGGL(kernel, dim3(groups + repack_groups(also)), dim3(256), 0, s, M, N, dy, lddy, z, ldz, dz,
                       dz_lo, lddz, act, sums, dbias, also, groups);
    return hipGetLastError();
}

hipError_t launch_sum_blocks(int blocks, int N, const float *sums, uint16_t *out, bool bf16, hipStream_t s)
{
    hipLaunchKernelGGL((bf16 ? sum_blocks_kernel<Brain16> : sum_blocks_kernel<Half16>), dim3((N + 31) / 32),
                       dim3(256), 0, s, blocks, N, sums, out);
    return hipGetLastError();
}

hipError_t launch_gate_grad(int M, int F, const uint16_t *dh, int lddh, const uint16_t *g, const uint16_t *u, int ldp,
                            const GateGrads &d, int ldd, int act, const Repack &q, bool bf16, hipStream_t s)
{
    Repack also = q;
    const unsigned groups = gate_groups(M, F);
    hipLaunchKernelGGL((bf16 ? gate_grad_kernel<Brain16> : gate_grad_kernel<Half16>), dim3(groups + repack_groups(also)),
                       dim3(256), 0, s, M, F, dh, lddh, g, u, ldp, d, ldd, act, also, groups,
                       gate_blocks(M, F));
    return hipGetLastError();
}

}  // namespace dgor
