// Layer norm and its backward pass.
//
//   mean = sum_j x_j / N,  rstd = 1 / sqrt(sum_j (x_j - mean)^2 / N + eps),
//   y_j = (x_j - mean) rstd w_j + b_j;
//   with xh_j = (x_j - mean) rstd and t_j = dy_j w_j:
//   dx_j = rstd (t_j - sum_i t_i / N - xh_j sum_i t_i xh_i / N),
//   dw_j = sum over rows of dy_j xh_j,  db_j = sum over rows of dy_j.
//
// Bound by memory.  A row is held in registers, eight elements of a thread
// at a time, so it is read once: rows of up to 1024 elements by one wavefront
// (four rows a workgroup, no barrier), up to 16384 by a workgroup of 256.
// The variance is the second pass over the registers, around the mean, so
// it loses nothing where the mean is large.  Longer rows are read again for
// each pass (the second read comes from the caches).
// The weight gradients: a workgroup takes every gridDim-th row and keeps its
// columns' sums in registers, so dy and x are read once for dx, dw and db
// together; the workgroups' sums are added in a fixed order by a second
// kernel.
#include "common.h"
#include "linear.h"

namespace dgor {
namespace {

struct Single {
    using T = float;
    static __device__ __forceinline__ void load8(const float *p, int n, float (&f)[8]) { load8_f32(p, n, f); }
    static __device__ __forceinline__ void store8(float *p, int n, const float (&f)[8]) { store8_f32(p, n, f); }
    static __device__ __forceinline__ float down(float f) { return f; }
};
template <class Fmt>
struct Short {
    using T = uint16_t;
    static __device__ __forceinline__ void load8(const uint16_t *p, int n, float (&f)[8])
    {
        unpack8<Fmt>(load8_16(p, n), f);
    }
    static __device__ __forceinline__ void store8(uint16_t *p, int n, const float (&f)[8])
    {
        store8_16(p, n, pack8<Fmt>(f));
    }
    static __device__ __forceinline__ uint16_t down(float f) { return Fmt::down(f); }
};

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int m = 32; m; m >>= 1)
        v += __shfl_xor(v, m);
    return v;
}

// The sums of a and b over the RT threads of a row, in every one of them.
// slots: 8 floats of LDS, not read since the last barrier.
template <int RT>
__device__ __forceinline__ void row_sum2(float &a, float &b, float *slots)
{
    a = wave_sum(a);
    b = wave_sum(b);
    if (RT == 64)
        return;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
        slots[wave] = a;
        slots[4 + wave] = b;
    }
    __syncthreads();
    a = (slots[0] + slots[1]) + (slots[2] + slots[3]);
    b = (slots[4] + slots[5]) + (slots[6] + slots[7]);
}

template <class X, class W, int RT, int V>
__global__ __launch_bounds__(256) void layer_norm_kernel(int M, int N, const typename X::T *__restrict__ x, int ldx,
                                                         const typename W::T *__restrict__ weight,
                                                         const typename W::T *__restrict__ bias, float eps,
                                                         typename X::T *__restrict__ y, int ldy,
                                                         float *__restrict__ mean_out, float *__restrict__ rstd_out)
{
    __shared__ float slots[2][8];
    constexpr int ROWS = 256 / RT;
    const int at = threadIdx.x % RT;
    // a row's two sums use a slot each, with a barrier between any write of a
    // slot and its last readers; with a row a wavefront there is no barrier
    for (long long row = blockIdx.x * ROWS + (RT == 64 ? (int)(threadIdx.x >> 6) : 0); row < M;
         row += (long long)gridDim.x * ROWS) {
        float v[V][8], sum = 0.f, none = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (at + RT * i);
            if (c < N)
                X::load8(x + (size_t)row * ldx + c, N - c, v[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (8 * (at + RT * i) < N)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum += v[i][e];   // elements past the row are zero
        row_sum2<RT>(sum, none, slots[0]);
        const float mean = sum / (float)N;
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (at + RT * i);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[i][e] -= mean;
                if (c + e < N)
                    sq = __builtin_fmaf(v[i][e], v[i][e], sq);
            }
        }
        row_sum2<RT>(sq, none, slots[1]);
        const float rstd = 1.f / sqrtf(sq / (float)N + eps);
        if (at == 0) {
            if (mean_out)
                mean_out[row] = mean;
            if (rstd_out)
                rstd_out[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (at + RT * i), n = N - c;
            if (n <= 0)
                break;
            float w[8], b[8];
            if (weight)
                W::load8(weight + c, n, w);
            if (bias)
                W::load8(bias + c, n, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = v[i][e] * rstd;
                v[i][e] = __builtin_fmaf(h, weight ? w[e] : 1.f, bias ? b[e] : 0.f);
            }
            X::store8(y + (size_t)row * ldy + c, n, v[i]);
        }
    }
}

// Rows longer than a workgroup's registers hold.
template <class X, class W>
__global__ __launch_bounds__(256) void layer_norm_long_kernel(int M, int N, const typename X::T *__restrict__ xs,
                                                              int ldx,
                                                              const typename W::T *__restrict__ weight,
                                                              const typename W::T *__restrict__ bias, float eps,
                                                              typename X::T *__restrict__ ys, int ldy,
                                                              float *__restrict__ mean_out,
                                                              float *__restrict__ rstd_out)
{
    __shared__ float slots[2][8];
    for (size_t row = blockIdx.x; row < (size_t)M; row += gridDim.x) {
        const typename X::T *x = xs + row * ldx;
        typename X::T *y = ys + row * ldy;
        float sum = 0.f, none = 0.f, sq = 0.f, v[8], w[8], b[8];
        for (int c = 8 * threadIdx.x; c < N; c += 2048) {
            X::load8(x + c, N - c, v);
            sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
        row_sum2<256>(sum, none, slots[0]);
        const float mean = sum / (float)N;
        for (int c = 8 * threadIdx.x; c < N; c += 2048) {
            X::load8(x + c, N - c, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < N)
                    sq = __builtin_fmaf(v[e] - mean, v[e] - mean, sq);
        }
        row_sum2<256>(sq, none, slots[1]);
        const float rstd = 1.f / sqrtf(sq / (float)N + eps);
        if (threadIdx.x == 0) {
            if (mean_out)
                mean_out[row] = mean;
            if (rstd_out)
                rstd_out[row] = rstd;
        }
        for (int c = 8 * threadIdx.x; c < N; c += 2048) {
            X::load8(x + c, N - c, v);
            if (weight)
                W::load8(weight + c, N - c, w);
            if (bias)
                W::load8(bias + c, N - c, b);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = __builtin_fmaf((v[e] - mean) * rstd, weight ? w[e] : 1.f, bias ? b[e] : 0.f);
            X::store8(y + c, N - c, v);
        }
    }
}

template <class X, class W, int RT, int V>
__global__ __launch_bounds__(256) void layer_norm_backward_kernel(
    int M, int N, const typename X::T *__restrict__ dy, int lddy, const typename X::T *__restrict__ x, int ldx,
    const typename W::T *__restrict__ weight, const float *__restrict__ mean, const float *__restrict__ rstd,
    typename X::T *__restrict__ dx, int lddx, float *__restrict__ sums)
{
    constexpr int ROWS = 256 / RT;
    __shared__ float slots[2][8];
    const int at = threadIdx.x % RT, sub = RT == 64 ? (int)(threadIdx.x >> 6) : 0;
    float w[V][8], dw[V][8], db[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (at + RT * i);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw[i][e] = db[i][e] = 0.f;
            w[i][e] = 1.f;
        }
        if (weight && c < N)
            W::load8(weight + c, N - c, w[i]);
    }
    const float inv = 1.f / (float)N;
    int turn = 0;
    // every wavefront of a workgroup that shares a row runs the same trips
    for (long long row = blockIdx.x * ROWS + sub; row < M; row += gridDim.x * ROWS, turn ^= 1) {
        float h[V][8], t[V][8], a = 0.f, b = 0.f;
        const float mu = mean[row], rs = rstd[row];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (at + RT * i);
            if (c < N) {
                X::load8(x + (size_t)row * ldx + c, N - c, h[i]);
                X::load8(dy + (size_t)row * lddy + c, N - c, t[i]);   // zero past the row
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    h[i][e] = t[i][e] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[i][e] = (h[i][e] - mu) * rs;
                dw[i][e] = __builtin_fmaf(t[i][e], h[i][e], dw[i][e]);
                db[i][e] += t[i][e];
                t[i][e] *= w[i][e];
                a += t[i][e];
                b = __builtin_fmaf(t[i][e], h[i][e], b);
            }
        row_sum2<RT>(a, b, slots[turn]);
        a *= inv;
        b *= inv;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (at + RT * i);
            if (c < N) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    t[i][e] = rs * (t[i][e] - a - h[i][e] * b);
                X::store8(dx + (size_t)row * lddx + c, N - c, t[i]);
            }
        }
    }
    if (!sums)
        return;
    float *out = sums + (size_t)blockIdx.x * 2 * N;
    if constexpr (RT == 64) {
        // the four wavefronts' sums, added in LDS in their order
        __shared__ float part[3][V * 512];
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            float(&mine)[V][8] = pass ? db : dw;
            __syncthreads();
            if (sub > 0)
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        part[sub - 1][(i * 8 + e) * 64 + at] = mine[i][e];
            __syncthreads();
            if (sub == 0)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int c = 8 * (at + RT * i);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int k = (i * 8 + e) * 64 + at;
                        mine[i][e] = ((mine[i][e] + part[0][k]) + part[1][k]) + part[2][k];
                    }
                    if (c < N)
                        store8_f32(out + pass * N + c, N - c, mine[i]);
                }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = 8 * (at + RT * i);
            if (c < N) {
                store8_f32(out + c, N - c, dw[i]);
                store8_f32(out + N + c, N - c, db[i]);
            }
        }
    }
}

// Rows longer than a workgroup's registers hold: dx by the row, and the
// weight gradients' sums by blocks of rows.
template <class X, class W>
__global__ __launch_bounds__(256) void layer_norm_backward_long_kernel(
    int M, int N, const typename X::T *__restrict__ dys, int lddy, const typename X::T *__restrict__ xs, int ldx,
    const typename W::T *__restrict__ weight, const float *__restrict__ mean, const float *__restrict__ rstd,
    typename X::T *__restrict__ dxs, int lddx)
{
    __shared__ float slots[2][8];
    int turn = 0;
    for (size_t row = blockIdx.x; row < (size_t)M; row += gridDim.x, turn ^= 1) {
        const typename X::T *dy = dys + row * lddy, *x = xs + row * ldx;
        typename X::T *dx = dxs + row * lddx;
        const float mu = mean[row], rs = rstd[row];
        float a = 0.f, b = 0.f, h[8], t[8], w[8];
        auto fetch = [&](int c) {
            X::load8(x + c, N - c, h);
            X::load8(dy + c, N - c, t);
            if (weight)
                W::load8(weight + c, N - c, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[e] = (h[e] - mu) * rs;
                t[e] *= weight ? w[e] : 1.f;
            }
        };
        for (int c = 8 * threadIdx.x; c < N; c += 2048) {
            fetch(c);
            float p = 0.f, q = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p += t[e];
                q = __builtin_fmaf(t[e], h[e], q);
            }
            a += p;
            b += q;
        }
        row_sum2<256>(a, b, slots[turn]);
        a /= (float)N;
        b /= (float)N;
        for (int c = 8 * threadIdx.x; c < N; c += 2048) {
            fetch(c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t[e] = rs * (t[e] - a - h[e] * b);
            X::store8(dx + c, N - c, t);
        }
    }
}

template <class X>
__global__ __launch_bounds__(256) void layer_norm_sums_kernel(int M, int N, const typename X::T *__restrict__ dy,
                                                              int lddy, const typename X::T *__restrict__ x, int ldx,
                                                              const float *__restrict__ mean,
                                                              const float *__restrict__ rstd, int rows,
                                                              float *__restrict__ sums)
{
    const int c = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (c >= N)
        return;
    const int n = N - c;
    const long long r0 = (long long)blockIdx.y * rows, r1 = min(r0 + rows, (long long)M);
    float dw[8] = {}, db[8] = {}, h[8], t[8];
    for (long long row = r0; row < r1; ++row) {
        X::load8(x + (size_t)row * ldx + c, n, h);
        X::load8(dy + (size_t)row * lddy + c, n, t);
        const float mu = mean[row], rs = rstd[row];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw[e] = __builtin_fmaf(t[e], (h[e] - mu) * rs, dw[e]);
            db[e] += t[e];
        }
    }
    float *out = sums + (size_t)blockIdx.y * 2 * N;
    store8_f32(out + c, n, dw);
    store8_f32(out + N + c, n, db);
}

// dw, db = the sums of `blocks` rows of 2 N, in a fixed order: 32 columns x 8
// threads over the blocks.
template <class W>
__global__ __launch_bounds__(256) void layer_norm_join_kernel(int blocks, int N, const float *__restrict__ sums,
                                                              typename W::T *__restrict__ dweight,
                                                              typename W::T *__restrict__ dbias)
{
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, b8 = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < 2LL * N)
#pragma unroll 4
        for (int b = b8; b < blocks; b += 8)
            s += sums[(size_t)b * 2 * N + c];
    part[b8][lane] = s;
    __syncthreads();
    if (b8 || c >= 2LL * N)
        return;
    s = ((part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane])) +
        ((part[4][lane] + part[5][lane]) + (part[6][lane] + part[7][lane]));
    if (c < N) {
        if (dweight)
            dweight[c] = W::down(s);
    } else if (dbias) {
        dbias[c - N] = W::down(s);
    }
}

constexpr int kMaxHeld = 16384;   // longest row that a workgroup holds
constexpr int kBackwardGroups = 512;   // workgroups of the backward kernel: two a compute unit

struct NormArgs {
    int M, N;
    const void *dy, *x, *weight, *bias;
    int lddy, ldx, ldout;
    float eps;
    void *out;
    float *mean, *rstd, *sums;
    int blocks;
    void *dweight, *dbias;
};

// A grid's workgroups: one for each row (or four rows) up to a million, whose
// loops then take the rest.
unsigned most(long long rows) { return (unsigned)(rows < (1 << 20) ? rows : (1 << 20)); }

template <class X, class W, int RT, int V>
hipError_t forward_as(const NormArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL((layer_norm_kernel<X, W, RT, V>), dim3(most(((long long)a.M + 256 / RT - 1) / (256 / RT))), dim3(256), 0, s, a.M,
                       a.N, (const typename X::T *)a.x, a.ldx, (const typename W::T *)a.weight,
                       (const typename W::T *)a.bias, a.eps, (typename X::T *)a.out, a.ldout, a.mean, a.rstd);
    return hipGetLastError();
}

template <class X, class W>
hipError_t forward(const NormArgs &a, hipStream_t s)
{
    if (a.N <= 512)
        return forward_as<X, W, 64, 1>(a, s);
    if (a.N <= 1024)
        return forward_as<X, W, 64, 2>(a, s);
    if (a.N <= 2048)
        return forward_as<X, W, 256, 1>(a, s);
    if (a.N <= 4096)
        return forward_as<X, W, 256, 2>(a, s);
    if (a.N <= 8192)
        return forward_as<X, W, 256, 4>(a, s);
    if (a.N <= kMaxHeld)
        return forward_as<X, W, 256, 8>(a, s);
    hipLaunchKernelGGL((layer_norm_long_kernel<X, W>), dim3(most(a.M)), dim3(256), 0, s, a.M, a.N, (const typename X::T *)a.x,
                       a.ldx, (const typename W::T *)a.weight, (const typename W::T *)a.bias, a.eps,
                       (typename X::T *)a.out, a.ldout, a.mean, a.rstd);
    return hipGetLastError();
}

template <class X, class W, int RT, int V>
hipError_t backward_as(const NormArgs &a, hipStream_t s)
{
    hipLaunchKernelGGL((layer_norm_backward_kernel<X, W, RT, V>), dim3(a.blocks), dim3(256), 0, s, a.M, a.N,
                       (const typename X::T *)a.dy, a.lddy, (const typename X::T *)a.x, a.ldx,
                       (const typename W::T *)a.weight, a.mean, a.rstd, (typename X::T *)a.out, a.ldout, a.sums);
    return hipGetLastError();
}

template <class X, class W>
hipError_t backward(const NormArgs &a, hipStream_t s)
{
    hipError_t err;
    if (a.N <= 512)
        err = backward_as<X, W, 64, 1>(a, s);
    else if (a.N <= 1024)
        err = backward_as<X, W, 64, 2>(a, s);
    else if (a.N <= 2048)
        err = backward_as<X, W, 256, 1>(a, s);
    else if (a.N <= 4096)
        err = backward_as<X, W, 256, 2>(a, s);
    else if (a.N <= 8192)
        err = backward_as<X, W, 256, 4>(a, s);
    else if (a.N <= kMaxHeld)
        err = backward_as<X, W, 256, 8>(a, s);
    else {
        hipLaunchKernelGGL((layer_norm_backward_long_kernel<X, W>), dim3(most(a.M)), dim3(256), 0, s, a.M, a.N,
                           (const typename X::T *)a.dy, a.lddy, (const typename X::T *)a.x, a.ldx,
                           (const typename W::T *)a.weight, a.mean, a.rstd, (typename X::T *)a.out, a.ldout);
        err = hipGetLastError();
        if (err == hipSuccess && a.sums) {
            hipLaunchKernelGGL((layer_norm_sums_kernel<X>), dim3((a.N + 2047) / 2048, a.blocks), dim3(256), 0, s, a.M,
                               a.N, (const typename X::T *)a.dy, a.lddy, (const typename X::T *)a.x, a.ldx, a.mean,
                               a.rstd, (a.M + a.blocks - 1) / a.blocks, a.sums);
            err = hipGetLastError();
        }
    }
    if (err != hipSuccess || !a.sums)
        return err;
    hipLaunchKernelGGL((layer_norm_join_kernel<W>), dim3((unsigned)((2LL * a.N + 31) / 32)), dim3(256), 0, s, a.blocks,
                       a.N, a.sums, (typename W::T *)a.dweight, (typename W::T *)a.dbias);
    return hipGetLastError();
}

enum class Type { F32, F16, BF16 };

template <class F>
hipError_t dispatch(Type t, bool weight_f32, F f)
{
    if (t == Type::F32)
        return f(Single{}, Single{});
    if (t == Type::F16)
        return weight_f32 ? f(Short<Half16>{}, Single{}) : f(Short<Half16>{}, Short<Half16>{});
    return weight_f32 ? f(Short<Brain16>{}, Single{}) : f(Short<Brain16>{}, Short<Brain16>{});
}

int check(const gemm_layer_norm_params *p)
{
    if (!p)
        return GEMM_ERR_NULL_PTR;
    if (p->M < 0 || p->N < 0 || !(p->eps >= 0.f))
        return GEMM_ERR_INVALID_DIM;
    const int least = p->N > 1 ? p->N : 1;
    if (p->ldx < least || p->ldy < least)
        return GEMM_ERR_INVALID_LAYOUT;
    return GEMM_OK;
}

// Workgroups of the backward kernel, each with its 2 N sums: no more than
// there are rows for.
int backward_blocks(int M, int N)
{
    const int rows = N <= 1024 ? 4 : 1;
    const int want = M / rows + (M % rows != 0);
    return want < kBackwardGroups ? want : kBackwardGroups;
}

int run_forward(Type t, const gemm_layer_norm_params *p, const void *x, const void *weight, const void *bias, void *y,
                float *mean, float *rstd, void *stream)
{
    const int rc = check(p);
    if (rc != GEMM_OK)
        return rc;
    if (p->M == 0 || p->N == 0)
        return GEMM_OK;
    if (!x || !y)
        return GEMM_ERR_NULL_PTR;
    const int dev = device_status();
    if (dev != GEMM_OK)
        return dev;
    NormArgs a{};
    a.M = p->M, a.N = p->N, a.x = x, a.weight = weight, a.bias = bias, a.ldx = p->ldx, a.ldout = p->ldy;
    a.eps = p->eps, a.out = y, a.mean = mean, a.rstd = rstd;
    const hipError_t err = dispatch(t, p->weight_f32 != 0, [&](auto X, auto W) {
        return forward<decltype(X), decltype(W)>(a, (hipStream_t)stream);
    });
    return err == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int run_backward(Type t, const gemm_layer_norm_params *p, const void *dy, const void *x, const void *weight,
                 const float *mean, const float *rstd, void *dx, void *dweight, void *dbias, void *ws,
                 size_t ws_bytes, void *stream)
{
    int rc = check(p);
    if (rc != GEMM_OK)
        return rc;
    if (p->lddx < (p->N > 1 ? p->N : 1))
        return GEMM_ERR_INVALID_LAYOUT;
    if (p->N == 0)
        return GEMM_OK;
    if (p->M > 0 && (!dy || !x || !mean || !rstd || !dx))
        return GEMM_ERR_NULL_PTR;
    NormArgs a{};
    a.M = p->M, a.N = p->N, a.dy = dy, a.x = x, a.weight = weight, a.lddy = p->ldy, a.ldx = p->ldx;
    a.ldout = p->lddx, a.out = dx, a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);
    a.dweight = dweight, a.dbias = dbias;
    a.blocks = backward_blocks(p->M, p->N);
    const bool grads = dweight || dbias, empty = p->M == 0;   // no rows: the weight gradients are empty sums
    if (grads && !empty) {
        if (!ws || ((uintptr_t)ws & 255) || ws_bytes < (size_t)a.blocks * 2 * p->N * sizeof(float))
            return GEMM_ERR_WORKSPACE;
        a.sums = (float *)ws;
    }
    if (empty && !grads)
        return GEMM_OK;
    const int dev = device_status();
    if (dev != GEMM_OK)
        return dev;
    const hipError_t err = dispatch(t, p->weight_f32 != 0, [&](auto X, auto W) {
        using WT = typename decltype(W)::T;
        if (empty) {
            hipLaunchKernelGGL((layer_norm_join_kernel<decltype(W)>), dim3((unsigned)((2LL * a.N + 31) / 32)),
                               dim3(256), 0, (hipStream_t)stream, 0, a.N, a.sums, (WT *)dweight, (WT *)dbias);
            return hipGetLastError();
        }
        return backward<decltype(X), decltype(W)>(a, (hipStream_t)stream);
    });
    return err == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace
}  // namespace dgor

extern "C" {

int gemm_layer_norm_f32(const gemm_layer_norm_params *params, const float *x, const float *weight, const float *bias,
                        float *y, float *mean, float *rstd, void *stream)
{
    return dgor::run_forward(dgor::Type::F32, params, x, weight, bias, y, mean, rstd, stream);
}
int gemm_layer_norm_f16(const gemm_layer_norm_params *params, const uint16_t *x, const void *weight, const void *bias,
                        uint16_t *y, float *mean, float *rstd, void *stream)
{
    return dgor::run_forward(dgor::Type::F16, params, x, weight, bias, y, mean, rstd, stream);
}
int gemm_layer_norm_bf16(const gemm_layer_norm_params *params, const uint16_t *x, const void *weight,
                         const void *bias, uint16_t *y, float *mean, float *rstd, void *stream)
{
    return dgor::run_forward(dgor::Type::BF16, params, x, weight, bias, y, mean, rstd, stream);
}

int gemm_layer_norm_backward_workspace(const gemm_layer_norm_params *params, size_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_NULL_PTR;
    const int rc = dgor::check(params);
    if (rc == GEMM_OK)
        *bytes = (size_t)dgor::backward_blocks(params->M, params->N) * 2 * params->N * sizeof(float);
    return rc;
}
int gemm_layer_norm_backward_f32(const gemm_layer_norm_params *params, const float *dy, const float *x,
                                 const float *weight, const float *mean, const float *rstd, float *dx,
                                 float *dweight, float *dbias, void *workspace, size_t workspace_bytes, void *stream)
{
    return dgor::run_backward(dgor::Type::F32, params, dy, x, weight, mean, rstd, dx, dweight, dbias, workspace,
                              workspace_bytes, stream);
}
int gemm_layer_norm_backward_f16(const gemm_layer_norm_params *params, const uint16_t *dy, const uint16_t *x,
                                 const void *weight, const float *mean, const float *rstd, uint16_t *dx, void *dweight,
                                 void *dbias, void *workspace, size_t workspace_bytes, void *stream)
{
    return dgor::run_backward(dgor::Type::F16, params, dy, x, weight, mean, rstd, dx, dweight, dbias, workspace,
                              workspace_bytes, stream);
}
int gemm_layer_norm_backward_bf16(const gemm_layer_norm_params *params, const uint16_t *dy, const uint16_t *x,
                                  const void *weight, const float *mean, const float *rstd, uint16_t *dx,
                                  void *dweight, void *dbias, void *workspace, size_t workspace_bytes, void *stream)
{
    return dgor::run_backward(dgor::Type::BF16, params, dy, x, weight, mean, rstd, dx, dweight, dbias, workspace,
                              workspace_bytes, stream);
}

}  // extern "C"
