// Layer norm and its backward pass.
//
//   mean = sum_j x_j / N,  rstd = 1 / sqrt(sum_j (x_j - mean)^2 / N + eps),
//   y_j = (x_j - mean) rstd w_j + b_j;
//   with xh_j = (x_j - mean) rstd and t_j = dy_j w_j:
//   dx_j = rstd (t_j - sum_i t_i / N - xh_j sum_i t_i xh_i / N),
//   dw_j = sum over rows of dy_j xh_j,  db_j = sum over rows of dy_j.
//
// Bound by memory.  A row is held in registers, eight elements of a thread
// at a time, so it is read once: in the forward pass rows of up to 1024
// elements by one wavefront (four rows a workgroup, no barrier), up to 16384 by
// a workgroup of 256 to 1024; all of a row's loads, the weights' among them, are
// issued before the first sum.  Sums within a wavefront are shifts on the
// vector ALUs.  The variance is the second pass over the registers, around the
// mean, so it loses nothing where the mean is large.  Longer rows are read
// again for each pass (the second read comes from the caches).
// 8192 x 4096 BF16: 23.3 us, 5.8 TB/s (26.4 for torch's copy of it); with sums
// through LDS shuffles and the weights loaded after them it took 37.
// The weight gradients: a workgroup, one for each compute unit, takes every
// gridDim-th rows and keeps its columns' sums in registers, so dy and x are
// read once for dx, dw and db together; the workgroups' sums are added in a
// fixed order by a second kernel.  8192 x 4096 BF16: 42 us, 4.8 TB/s.
#include "common.h"
#include "linear.h"

namespace dgor {
namespace {

struct Single {
    using T = float;
    // eight elements as they are loaded, and opened
    struct Raw {
        float f[8];
    };
    static __device__ __forceinline__ Raw fetch(const float *p, int n)
    {
        Raw r;
        load8_f32(p, n, r.f);
        return r;
    }
    static __device__ __forceinline__ void open(const Raw &r, float (&f)[8])
    {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = r.f[e];
    }
    // makes the value one that the compiler has not seen
    static __device__ __forceinline__ void renew(Raw &r)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            asm volatile("" : "+v"(r.f[e]));
    }
    static __device__ __forceinline__ void load8(const float *p, int n, float (&f)[8]) { load8_f32(p, n, f); }
    static __device__ __forceinline__ void store8(float *p, int n, const float (&f)[8]) { store8_f32(p, n, f); }
    static __device__ __forceinline__ float down(float f) { return f; }
};
template <class Fmt>
struct Short {
    using T = uint16_t;
    using Raw = u32x4;
    static __device__ __forceinline__ Raw fetch(const uint16_t *p, int n) { return load8_16(p, n); }
    static __device__ __forceinline__ void open(const Raw &r, float (&f)[8]) { unpack8<Fmt>(r, f); }
    static __device__ __forceinline__ void renew(Raw &r) { asm volatile("" : "+v"(r)); }
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

// A wavefront's sum, in every lane: four shifts within rows of 16 lanes, two
// across them, all on the vector ALUs.
template <int CONTROL, int ROWS>
__device__ __forceinline__ float add_shifted(float v)
{
    const int t = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CONTROL, ROWS, 0xf, false);
    return v + __builtin_bit_cast(float, t);
}
__device__ __forceinline__ float wave_sum(float v)
{
    v = add_shifted<0x111, 0xf>(v);   // row_shr:1, 2, 4, 8; lanes without a source add zero
    v = add_shifted<0x112, 0xf>(v);
    v = add_shifted<0x114, 0xf>(v);
    v = add_shifted<0x118, 0xf>(v);
    v = add_shifted<0x142, 0xa>(v);   // row_bcast:15 into rows 1 and 3
    v = add_shifted<0x143, 0xc>(v);   // row_bcast:31 into rows 2 and 3
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// The sum of a over the RT threads of a row, in every one of them.
// slots: a float of LDS for each of the row's wavefronts, not read since the
// last barrier.
template <int RT>
__device__ __forceinline__ float row_sum(float a, float *slots)
{
    a = wave_sum(a);
    if (RT == 64)
        return a;
    if ((threadIdx.x & 63) == 0)
        slots[threadIdx.x % RT / 64] = a;
    __syncthreads();
    a = slots[0];
#pragma unroll
    for (int i = 1; i < RT / 64; ++i)
        a += slots[i];
    return a;
}

// The sums of a and b likewise; slots: two floats a wavefront.
template <int RT>
__device__ __forceinline__ void row_sum2(float &a, float &b, float *slots)
{
    a = wave_sum(a);
    b = wave_sum(b);
    if (RT == 64)
        return;
    const int wave = threadIdx.x % RT / 64;
    if ((threadIdx.x & 63) == 0) {
        slots[2 * wave] = a;
        slots[2 * wave + 1] = b;
    }
    __syncthreads();
    a = slots[0];
    b = slots[1];
#pragma unroll
    for (int i = 1; i < RT / 64; ++i) {
        a += slots[2 * i];
        b += slots[2 * i + 1];
    }
}

// How a row ends.  kCut: the last unit is the row's last eight elements, which
// two threads then both have: they count in the sums of the first, and both
// write what they come to.  So no access branches on the row's end (masked
// loads of single elements made 8192 x 4093 take twice as long as 8192 x 4096).
// kNarrow: rows shorter than a unit.
enum RowEnd { kWhole, kCut, kNarrow };

// A unit's column, how many elements from it to load, and how many of those
// belong to the unit before.
template <RowEnd END>
struct Unit {
    int c, n, shared;
    __device__ __forceinline__ Unit(int at, int N)
        : c(END == kCut ? min(at, N - 8) : at), n(END == kNarrow ? N - at : 8), shared(at - c)
    {
    }
    // whether element e is this unit's to count
    __device__ __forceinline__ bool counts(int e) const
    {
        return END == kWhole || (END == kCut ? e >= shared : e < n);
    }
};

constexpr int group_threads(int rt) { return rt > 256 ? rt : 256; }
template <class X, class W, int RT, int V, RowEnd END>
__global__ __launch_bounds__(group_threads(RT)) void layer_norm_kernel(int M, int N, const typename X::T *__restrict__ x, int ldx,
                                                         const typename W::T *__restrict__ weight,
                                                         const typename W::T *__restrict__ bias, float eps,
                                                         typename X::T *__restrict__ y, int ldy,
                                                         float *__restrict__ mean_out, float *__restrict__ rstd_out)
{
    __shared__ float slots[2][RT / 64];
    constexpr int ROWS = group_threads(RT) / RT;
    const int at = threadIdx.x % RT;
    // a row's two sums use a slot each, with a barrier between any write of a
    // slot and its last readers; with a row a wavefront there is no barrier
    for (long long row = blockIdx.x * ROWS + (RT == 64 ? (int)(threadIdx.x >> 6) : 0); row < M;
         row += (long long)gridDim.x * ROWS) {
        // all of the row's loads first, the weights' among them
        typename X::Raw xr[V];
        typename W::Raw wr[V], br[V];
        float v[V][8], sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (8 * (at + RT * i) >= N)
                continue;
            const Unit<END> u(8 * (at + RT * i), N);
            xr[i] = X::fetch(x + (size_t)row * ldx + u.c, u.n);
            if (weight)
                wr[i] = W::fetch(weight + u.c, u.n);
            if (bias)
                br[i] = W::fetch(bias + u.c, u.n);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (8 * (at + RT * i) >= N)
                continue;
            const Unit<END> u(8 * (at + RT * i), N);
            X::open(xr[i], v[i]);
            float t[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t[e] = u.counts(e) ? v[i][e] : 0.f;
            sum += ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
        }
        const float mean = row_sum<RT>(sum, slots[0]) / (float)N;
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (8 * (at + RT * i) >= N)
                continue;
            const Unit<END> u(8 * (at + RT * i), N);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[i][e] -= mean;
                sq = u.counts(e) ? __builtin_fmaf(v[i][e], v[i][e], sq) : sq;
            }
        }
        const float rstd = 1.f / sqrtf(row_sum<RT>(sq, slots[1]) / (float)N + eps);
        if (at == 0) {
            if (mean_out)
                mean_out[row] = mean;
            if (rstd_out)
                rstd_out[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (8 * (at + RT * i) >= N)
                continue;
            const Unit<END> u(8 * (at + RT * i), N);
            float w[8], b[8];
            if (weight)
                W::open(wr[i], w);
            if (bias)
                W::open(br[i], b);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i][e] = __builtin_fmaf(v[i][e] * rstd, weight ? w[e] : 1.f, bias ? b[e] : 0.f);
            X::store8(y + (size_t)row * ldy + u.c, u.n, v[i]);
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
    __shared__ float slots[2][4];
    for (size_t row = blockIdx.x; row < (size_t)M; row += gridDim.x) {
        const typename X::T *x = xs + row * ldx;
        typename X::T *y = ys + row * ldy;
        float sum = 0.f, sq = 0.f, v[8], w[8], b[8];
        for (int c = 8 * threadIdx.x; c < N; c += 2048) {
            X::load8(x + c, N - c, v);
            sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
        const float mean = row_sum<256>(sum, slots[0]) / (float)N;
        for (int c = 8 * threadIdx.x; c < N; c += 2048) {
            X::load8(x + c, N - c, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < N)
                    sq = __builtin_fmaf(v[e] - mean, v[e] - mean, sq);
        }
        const float rstd = 1.f / sqrtf(row_sum<256>(sq, slots[1]) / (float)N + eps);
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

// G rows at a time, by RT threads each, 1024 in all; a workgroup takes rows
// blockIdx.x G + g, then gridDim.x G further on.  With one unit a thread, the
// next row's loads are issued before a row is worked on; with two the
// registers do not hold them, nor the opened values across the row's sums: a
// row is opened again behind them.  The groups' sums of dw and db meet in LDS,
// halves of the groups at a time in a fixed order; they go to
// sums[block][2][N] or, with one workgroup, straight to dweight and dbias.
template <class X, class W, int RT, int V, int G, RowEnd END>
__global__ __launch_bounds__(RT * G) void layer_norm_backward_kernel(
    int M, int N, const typename X::T *__restrict__ dy, int lddy, const typename X::T *__restrict__ x, int ldx,
    const typename W::T *__restrict__ weight, const float *__restrict__ mean, const float *__restrict__ rstd,
    typename X::T *__restrict__ dx, int lddx, float *__restrict__ sums, typename W::T *__restrict__ dweight,
    typename W::T *__restrict__ dbias)
{
    __shared__ float slots[2][RT / 32 * G];
    const int at = threadIdx.x % RT, group = threadIdx.x / RT;
    typename W::Raw wr[V];
    float dw[V][8], db[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            dw[i][e] = db[i][e] = 0.f;
        const Unit<END> u(8 * (at + RT * i), N);
        if (weight && 8 * (at + RT * i) < N)
            wr[i] = W::fetch(weight + u.c, u.n);
    }
    typename X::Raw xr[V], tr[V];
    float mu = 0.f, rs = 0.f;
    auto fetch = [&](long long row) {
        if (row >= M)
            return;
        mu = mean[row];
        rs = rstd[row];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Unit<END> u(8 * (at + RT * i), N);
            if (8 * (at + RT * i) < N) {
                xr[i] = X::fetch(x + (size_t)row * ldx + u.c, u.n);
                tr[i] = X::fetch(dy + (size_t)row * lddy + u.c, u.n);
            }
        }
    };
    // unit i's normalised values, and dy
    auto open = [&](int i, float (&h)[8], float (&t)[8]) {
        X::open(xr[i], h);
        X::open(tr[i], t);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            h[e] = (h[e] - mu) * rs;
    };
    auto weigh = [&](int i, float (&t)[8]) {
        if (!weight)
            return;
        float w[8];
        W::open(wr[i], w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            t[e] *= w[e];
    };
    const float inv = 1.f / (float)N;
    const long long step = (long long)gridDim.x * G;
    if (V == 1)
        fetch((long long)blockIdx.x * G + group);
    int turn = 0;
    // every wavefront of the workgroup runs the same trips
    for (long long first = (long long)blockIdx.x * G; first < M; first += step, turn ^= 1) {
        const long long row = first + group;
        constexpr int KEPT = V == 1 ? 1 : 0;
        float hk[KEPT + 1][8], tk[KEPT + 1][8], a = 0.f, b = 0.f;
        if (V > 1)
            fetch(row);
        const float rs_row = rs;
        if (row < M)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (8 * (at + RT * i) >= N)
                    continue;
                const Unit<END> u(8 * (at + RT * i), N);
                float h[8], t[8];
                open(i, h, t);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dw[i][e] = __builtin_fmaf(t[e], h[e], dw[i][e]);
                    db[i][e] += t[e];
                }
                weigh(i, t);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    a = u.counts(e) ? a + t[e] : a;
                    b = u.counts(e) ? __builtin_fmaf(t[e], h[e], b) : b;
                    if (V == 1)
                        hk[0][e] = h[e], tk[0][e] = t[e];
                }
            }
        if (V == 1)
            fetch(row + step);
        row_sum2<RT>(a, b, slots[turn] + RT / 32 * group);
        a *= inv;
        b *= inv;
        if (row < M)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (8 * (at + RT * i) >= N)
                    continue;
                const Unit<END> u(8 * (at + RT * i), N);
                float h[8], t[8];
                if (V == 1) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        h[e] = hk[0][e], t[e] = tk[0][e];
                } else {
                    X::renew(xr[i]);   // or the compiler keeps the opened values
                    X::renew(tr[i]);
                    open(i, h, t);
                    weigh(i, t);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    t[e] = rs_row * (t[e] - a - h[e] * b);
                X::store8(dx + (size_t)row * lddx + u.c, u.n, t);
            }
    }
    if (!sums && !dweight && !dbias)
        return;
    if constexpr (G > 1) {
        __shared__ float part[G / 2][2][V * 8 * RT];
#pragma unroll
        for (int half = G / 2; half; half /= 2) {
            __syncthreads();   // the part's readers are done
            if (group >= half && group < 2 * half)
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        part[group - half][0][(i * 8 + e) * RT + at] = dw[i][e];
                        part[group - half][1][(i * 8 + e) * RT + at] = db[i][e];
                    }
            __syncthreads();
            if (group < half)
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dw[i][e] += part[group][0][(i * 8 + e) * RT + at];
                        db[i][e] += part[group][1][(i * 8 + e) * RT + at];
                    }
        }
        if (group)
            return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (8 * (at + RT * i) >= N)
            continue;
        const Unit<END> u(8 * (at + RT * i), N);
        if (sums) {
            float *out = sums + (size_t)blockIdx.x * 2 * N;
            store8_f32(out + u.c, u.n, dw[i]);
            store8_f32(out + N + u.c, u.n, db[i]);
        } else {
            if (dweight)
                W::store8(dweight + u.c, u.n, dw[i]);
            if (dbias)
                W::store8(dbias + u.c, u.n, db[i]);
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
    // every thread of the workgroup makes the same turns: more than one where the
    // grid is at its most
    for (long long first = (long long)blockIdx.x * 32; first < 2LL * N; first += (long long)gridDim.x * 32) {
        const long long c = first + lane;
        float s = 0.f;
        if (c < 2LL * N)
#pragma unroll 4
            for (int b = b8; b < blocks; b += 8)
                s += sums[(size_t)b * 2 * N + c];
        part[b8][lane] = s;
        __syncthreads();
        if (b8 == 0 && c < 2LL * N) {
            s = ((part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane])) +
                ((part[4][lane] + part[5][lane]) + (part[6][lane] + part[7][lane]));
            if (c < N) {
                if (dweight)
                    dweight[c] = W::down(s);
            } else if (dbias) {
                dbias[c - N] = W::down(s);
            }
        }
        __syncthreads();   // the sums' readers are done
    }
}

constexpr int kMaxHeld = 16384;   // longest row that a workgroup holds
// Longest row: a column a step of the long kernels (2048) past it is still an int.
constexpr int kMaxColumns = 0x7fffffff - 4095;
constexpr int kUnits = 256;       // compute units

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

// A grid's workgroups: one for each row (or four rows, or 32 columns) up to a
// million, whose loops then take the rest.
unsigned most(long long want) { return (unsigned)(want < (1 << 20) ? want : (1 << 20)); }

template <class X, class W, int RT, int V>
hipError_t forward_as(const NormArgs &a, hipStream_t s)
{
    constexpr int ROWS = group_threads(RT) / RT;
    const dim3 grid(most(((long long)a.M + ROWS - 1) / ROWS));
    const auto kernel = a.N % 8 == 0 ? layer_norm_kernel<X, W, RT, V, kWhole>
                        : a.N > 8    ? layer_norm_kernel<X, W, RT, V, kCut>
                                     : layer_norm_kernel<X, W, 64, 1, kNarrow>;   // of the shortest rows' form
    hipLaunchKernelGGL(kernel, grid, dim3(group_threads(RT)), 0, s, a.M, a.N, (const typename X::T *)a.x, a.ldx,
                       (const typename W::T *)a.weight, (const typename W::T *)a.bias, a.eps,
                       (typename X::T *)a.out, a.ldout, a.mean, a.rstd);
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
        return forward_as<X, W, 512, 2>(a, s);
    if (a.N <= kMaxHeld)
        return forward_as<X, W, 1024, 2>(a, s);
    hipLaunchKernelGGL((layer_norm_long_kernel<X, W>), dim3(most(a.M)), dim3(256), 0, s, a.M, a.N, (const typename X::T *)a.x,
                       a.ldx, (const typename W::T *)a.weight, (const typename W::T *)a.bias, a.eps,
                       (typename X::T *)a.out, a.ldout, a.mean, a.rstd);
    return hipGetLastError();
}

template <class X, class W, int RT, int V, int G>
hipError_t backward_as(const NormArgs &a, hipStream_t s)
{
    using WT = typename W::T;
    const auto kernel = a.N % 8 == 0 ? layer_norm_backward_kernel<X, W, RT, V, G, kWhole>
                        : a.N > 8    ? layer_norm_backward_kernel<X, W, RT, V, G, kCut>
                                     : layer_norm_backward_kernel<X, W, 64, 1, 16, kNarrow>;   // of the shortest rows' form
    hipLaunchKernelGGL(kernel, dim3(a.blocks), dim3(RT * G), 0, s, a.M, a.N, (const typename X::T *)a.dy, a.lddy,
                       (const typename X::T *)a.x, a.ldx, (const WT *)a.weight, a.mean, a.rstd,
                       (typename X::T *)a.out, a.ldout, a.sums, a.sums ? nullptr : (WT *)a.dweight,
                       a.sums ? nullptr : (WT *)a.dbias);
    return hipGetLastError();
}

// Rows that a workgroup of the backward kernel works on at once.
int rows_at_once(int N)
{
    return N <= 512 ? 16 : (N <= 1024 ? 8 : (N <= 2048 ? 4 : (N <= 4096 ? 2 : 1)));
}

template <class X, class W>
hipError_t backward(const NormArgs &a, hipStream_t s)
{
    hipError_t err;
    if (a.N <= 512)
        err = backward_as<X, W, 64, 1, 16>(a, s);
    else if (a.N <= 1024)
        err = backward_as<X, W, 128, 1, 8>(a, s);
    else if (a.N <= 2048)
        err = backward_as<X, W, 256, 1, 4>(a, s);
    else if (a.N <= 4096)
        err = backward_as<X, W, 512, 1, 2>(a, s);
    else if (a.N <= 8192)
        err = backward_as<X, W, 1024, 1, 1>(a, s);
    else if (a.N <= kMaxHeld)
        err = backward_as<X, W, 1024, 2, 1>(a, s);
    else {
        hipLaunchKernelGGL((layer_norm_backward_long_kernel<X, W>), dim3(most(a.M)), dim3(256), 0, s, a.M, a.N,
                           (const typename X::T *)a.dy, a.lddy, (const typename X::T *)a.x, a.ldx,
                           (const typename W::T *)a.weight, a.mean, a.rstd, (typename X::T *)a.out, a.ldout);
        err = hipGetLastError();
        if (err == hipSuccess && a.sums) {
            hipLaunchKernelGGL((layer_norm_sums_kernel<X>), dim3((a.N + 2047) / 2048, a.blocks), dim3(256), 0, s, a.M,
                               a.N, (const typename X::T *)a.dy, a.lddy, (const typename X::T *)a.x, a.ldx, a.mean,
                               a.rstd, a.M / a.blocks + (a.M % a.blocks != 0), a.sums);
            err = hipGetLastError();
        }
    }
    if (err != hipSuccess || !a.sums)
        return err;
    hipLaunchKernelGGL((layer_norm_join_kernel<W>), dim3(most((2LL * a.N + 31) / 32)), dim3(256), 0, s, a.blocks, a.N,
                       a.sums, (typename W::T *)a.dweight, (typename W::T *)a.dbias);
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

// (eps is the forward pass's)
int check(const gemm_layer_norm_params *p)
{
    if (!p)
        return GEMM_ERR_NULL_PTR;
    if (p->M < 0 || p->N < 0 || p->N > kMaxColumns)
        return GEMM_ERR_INVALID_DIM;
    const int least = p->N > 1 ? p->N : 1;
    if (p->ldx < least || p->ldy < least)
        return GEMM_ERR_INVALID_LAYOUT;
    return GEMM_OK;
}

// Workgroups of the backward kernel, each with its 2 N sums: one for each
// compute unit, no more than there are rows for, and a single one, whose sums
// need no joining, for up to four turns.
int backward_blocks(int M, int N)
{
    const int rows = rows_at_once(N);
    if (M <= 4 * rows && N <= kMaxHeld)
        return 1;
    const int want = M / rows + (M % rows != 0);
    return want < kUnits ? want : kUnits;
}
// Whether the sums of the weights' gradients pass through the workspace.
bool joined(int M, int N) { return backward_blocks(M, N) > 1 || N > kMaxHeld; }

int run_forward(Type t, const gemm_layer_norm_params *p, const void *x, const void *weight, const void *bias, void *y,
                float *mean, float *rstd, void *stream)
{
    const int rc = check(p);
    if (rc != GEMM_OK)
        return rc;
    if (!(p->eps >= 0.f))
        return GEMM_ERR_INVALID_DIM;
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
    if (grads && !empty && joined(p->M, p->N)) {
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
            hipLaunchKernelGGL((layer_norm_join_kernel<decltype(W)>), dim3(most((2LL * a.N + 31) / 32)), dim3(256), 0,
                               (hipStream_t)stream, 0, a.N, a.sums, (WT *)dweight, (WT *)dbias);
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
        *bytes = dgor::joined(params->M, params->N)
                     ? (size_t)dgor::backward_blocks(params->M, params->N) * 2 * params->N * sizeof(float)
                     : 0;
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
