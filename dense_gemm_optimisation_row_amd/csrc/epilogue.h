// What the dense-layer kernels do with a finished sum: bias, saved
// pre-activation, activation (or the gate's product), residual and the
// rounding to the output type.  Internal header.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm.h"

namespace dgor {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// The 16-bit input formats: conversion to and from binary32.
struct Half16 {
    static __device__ __forceinline__ float up(uint16_t h) { return (float)__builtin_bit_cast(_Float16, h); }
    // round to nearest even, overflow to infinity
    static __device__ __forceinline__ uint16_t down(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
    static __device__ __forceinline__ uint32_t down2(float a, float b)
    {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, f16x2));
    }
};
struct Brain16 {
    static __device__ __forceinline__ float up(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
    // round to nearest even
    static __device__ __forceinline__ uint16_t down(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
    static __device__ __forceinline__ uint32_t down2(float a, float b)
    {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
    }
};

// Vectors at their element's alignment: global memory takes 16-byte accesses
// at any element address, so rows of any length move eight elements at a time.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));

// Eight (or the first n, at least one) elements of a 16-bit array, the rest
// zero.  The single elements are all loaded, past n the last again, so that
// their loads are in flight together (masked, each waits for the one before:
// 15 us for a kernel of eight such rows a thread, 5 so).
__device__ __forceinline__ u32x4 load8_16(const uint16_t *p, int n)
{
    if (n >= 8)
        return *reinterpret_cast<const u32x4_at2 *>(p);
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        h[e] = p[e < n ? e : n - 1];
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = (2 * e < n ? h[2 * e] : 0u) | (2 * e + 1 < n ? h[2 * e + 1] << 16 : 0u);
    return v;
}
__device__ __forceinline__ void store8_16(uint16_t *p, int n, u32x4 v)
{
    if (n >= 8) {
        *reinterpret_cast<u32x4_at2 *>(p) = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n)
            p[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
}
// A 16-bit operand as its units are loaded: rows x cols, at least eight
// elements from its first to its last.
//
// A unit is eight elements of row r from column c, a multiple of 8; what is
// outside the matrix counts as zero.  load reads the unit from the nearest
// place where the matrix holds eight elements (of the row, or across rows
// shorter than a unit); settle, when the load has arrived, shifts it into
// place and clears what is outside.  The load has no branch, so that a
// wavefront's loads stay in flight together, and a unit inside the matrix
// needs no settling.
struct Operand {
    const uint16_t *p;
    int rows, cols;
    size_t ld;

    __device__ __forceinline__ size_t row_at(int r) const { return (size_t)min(r, rows - 1) * ld; }
    __device__ __forceinline__ size_t last() const { return (size_t)(rows - 1) * ld + cols - 8; }
    __device__ __forceinline__ u32x4 load(int r, int c) const
    {
        size_t at = row_at(r);
        if (cols >= 8)
            at += min(c, cols - 8);
        else
            at = min(at, last());
        return *reinterpret_cast<const u32x4_at2 *>(p + at);
    }
    __device__ __forceinline__ u32x4 settle(u32x4 v, int r, int c) const
    {
        int off;
        bool keep = r < rows;
        if (cols >= 8) {
            off = c - min(c, cols - 8);
            keep = keep && off < 8;
        } else {
            off = (int)(row_at(r) - min(row_at(r), last()));
            keep = keep && c == 0;
        }
        const uint32_t half = 16u * (off & 1), m2 = -(uint32_t)(off >> 1 & 1), m4 = -(uint32_t)(off >> 2 & 1);
        uint32_t d[8] = {v[0], v[1], v[2], v[3], 0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            d[i] = __builtin_amdgcn_alignbit(d[i + 1], d[i], half);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            d[i] = (d[i + 1] & m2) | (d[i] & ~m2);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = keep ? (d[i + 2] & m4) | (d[i] & ~m4) : 0u;
        if (cols < 8)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] &= 2 * i + 1 < cols ? ~0u : (2 * i < cols ? 0xffffu : 0u);
        return v;
    }
};

template <class Fmt>
__device__ __forceinline__ void unpack8(u32x4 v, float (&f)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = Fmt::up((uint16_t)(v[e >> 1] >> (16 * (e & 1))));
}
template <class Fmt>
__device__ __forceinline__ u32x4 pack8(const float (&f)[8])
{
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = Fmt::down2(f[2 * e], f[2 * e + 1]);
    return v;
}
// f as the sum of two bfloat16 terms, to 2^-17 of it (a binary16 value exactly).
// What has no finite higher term is that term alone.
__device__ __forceinline__ void pack8_terms(const float (&f)[8], u32x4 &hi, u32x4 &lo)
{
    float r[8];
    hi = pack8<Brain16>(f);
    unpack8<Brain16>(hi, r);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        r[e] = __builtin_isfinite(r[e]) ? f[e] - r[e] : 0.f;
    lo = pack8<Brain16>(r);
}
__device__ __forceinline__ void load8_f32(const float *p, int n, float (&f)[8])
{
    if (n >= 8) {
        const f32x4 a = *reinterpret_cast<const f32x4_at4 *>(p), b = *reinterpret_cast<const f32x4_at4 *>(p + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[e] = a[e];
            f[4 + e] = b[e];
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = p[e < n ? e : n - 1];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = e < n ? f[e] : 0.f;
}
__device__ __forceinline__ void store8_f32(float *p, int n, const float (&f)[8])
{
    if (n >= 8) {
        *reinterpret_cast<f32x4_at4 *>(p) = f32x4{f[0], f[1], f[2], f[3]};
        *reinterpret_cast<f32x4_at4 *>(p + 4) = f32x4{f[4], f[5], f[6], f[7]};
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n)
            p[e] = f[e];
}

// ---- activations, in binary32.  exp is the hardware's base-2 exponential
// (one unit in the last place; the scaled argument adds |z| 2^-24 relative);
// the logistic function's quotient the hardware reciprocal.  A large
// negative z gives exp = infinity and a quotient of exactly zero.
__device__ __forceinline__ float act_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f); }
__device__ __forceinline__ float logistic(float x) { return __builtin_amdgcn_rcpf(1.f + act_exp(-x)); }

// z held to [-m, m]; a NaN stays one.  The slopes saturate long before m, and
// stay finite at the largest finite z.
__device__ __forceinline__ float held(float z, float m) { return z > m ? m : (z < -m ? -m : z); }

// The normal distribution function and e^(-z^2/2).  The tail is
// erfc(x) = e^(-x^2) t P(t), t = 1 / (1 + 0.4 x), at x = |z| / sqrt(2), with P of
// degree 8 fitted to e^(x^2) erfc(x) / t in the relative error's maximum over all
// x >= 0 (least squares under weights that are multiplied by the error until it is
// level): 1.3e-7.  So the lower tail keeps its relative accuracy: in binary32
// all in all (8 + z^2) 2^-24, the z^2 from the exponential's rounded argument.
__device__ __forceinline__ float normal_cdf(float z, float &bell)
{
    const float x = fabsf(z) * 0.70710678118654752440f;
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.4f, x, 1.f));
    bell = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170368f);   // log2(e) / 2
    constexpr float P[9] = {0.225675866f, 0.225669608f, 0.207842514f,  0.168543816f, 0.141422912f,
                            -0.00558640156f, 0.169056848f, -0.182881624f, 0.0502565987f};
    float poly = P[8];
#pragma unroll
    for (int i = 7; i >= 0; --i)
        poly = __builtin_fmaf(poly, t, P[i]);
    const float tail = 0.5f * (t * poly) * bell;
    return z > 0.f ? 1.f - tail : tail;
}

constexpr float kTanhScale = 1.59576912160573071176f;   // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

__device__ __forceinline__ float activate(int act, float z)
{
    switch (act) {
    case GEMM_ACT_RELU: return z <= 0.f ? 0.f : z;
    case GEMM_ACT_GELU: {
        float bell;
        return z * normal_cdf(z, bell);
    }
    case GEMM_ACT_GELU_TANH: {   // z (1 + tanh(y)) / 2 = z logistic(2 y)
        const float c = held(z, 64.f);
        return z * logistic(kTanhScale * c * __builtin_fmaf(kTanhCubic * c, c, 1.f));
    }
    case GEMM_ACT_SILU: return z * logistic(z);
    default: return z;
    }
}

// The activation's value and slope.
__device__ __forceinline__ void activate_slope(int act, float z, float &value, float &slope)
{
    switch (act) {
    case GEMM_ACT_RELU:
        value = z <= 0.f ? 0.f : z;
        slope = z <= 0.f ? 0.f : 1.f;
        return;
    case GEMM_ACT_GELU: {
        float bell;
        const float c = held(z, 64.f), p = normal_cdf(c, bell);
        value = z * p;
        slope = __builtin_fmaf(c * 0.39894228040143267794f, bell, p);
        return;
    }
    case GEMM_ACT_GELU_TANH: {
        const float c = held(z, 64.f), s = logistic(kTanhScale * c * __builtin_fmaf(kTanhCubic * c, c, 1.f));
        value = z * s;
        slope = __builtin_fmaf(c * s * (1.f - s) * kTanhScale, __builtin_fmaf(3.f * kTanhCubic * c, c, 1.f), s);
        return;
    }
    case GEMM_ACT_SILU: {
        const float c = held(z, 128.f), s = logistic(c);
        value = z * s;
        slope = s * __builtin_fmaf(c, 1.f - s, 1.f);
        return;
    }
    default:
        value = z;
        slope = 1.f;
    }
}

// Where a finished tile goes.  Y is M x N in FP32 (y_f32), binary16 (y_f16, of
// products on bfloat16 terms) or the input format; the rest may be null.  Gated
// products have two sums an element and two saved pre-activations.
struct Epilogue {
    void *Y;
    const uint16_t *bias;
    const void *R;         // residual, in Y's format
    uint16_t *pre, *pre2;
    int ldy, ldr, ldp;
    int act, y_f32, y_f16;
};

// The bias of eight neighbouring columns, n of them inside the matrix.
template <class Fmt>
__device__ __forceinline__ void load_bias(const Epilogue &e, int col, int n, float (&b)[8])
{
    u32x4 v = {0u, 0u, 0u, 0u};
    if (e.bias)
        v = load8_16(e.bias + col, n);
    unpack8<Fmt>(v, b);
}

// Eight neighbouring outputs (n of them inside the matrix) of each of the rows
// row, row + step, ... below M: v the sums, u the up projection's (gated only).
// The residual is read by the lane that writes the same elements of Y, so Y
// may be the residual itself; all rows' residuals are read before the first
// row is written, so that their loads are in flight together.  WHOLE: n is 8
// for every lane, so no access branches on it.  ACT: the activation, or
// kAnyActivation for e's.  bias: zeros without one (a sum is never -0: adding
// them changes nothing).
constexpr int kAnyActivation = -1;
template <class Fmt, bool GATED, bool WHOLE, int ACT, int ROWS>
__device__ __forceinline__ void emit_rows(const Epilogue &e, int row, int step, int M, int col, int inside,
                                          float (&v)[ROWS][8], const float (&u)[ROWS][8], const float (&bias)[8])
{
    const int n = WHOLE ? 8 : inside;
    float r[ROWS][8];
    if (!GATED && e.R) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int at = row + i * step;
            const size_t ra = (size_t)(at < M ? at : row) * e.ldr + col;
            if (e.y_f32)
                load8_f32((const float *)e.R + ra, n, r[i]);
            else
                unpack8<Fmt>(load8_16((const uint16_t *)e.R + ra, n), r[i]);
        }
    }
    if (!GATED)
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int c = 0; c < 8; ++c)
                v[i][c] += bias[c];
    if (e.pre) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (row + i * step < M) {
                const size_t at = (size_t)(row + i * step) * e.ldp + col;
                store8_16(e.pre + at, n, pack8<Fmt>(v[i]));
                if (GATED)
                    store8_16(e.pre2 + at, n, pack8<Fmt>(u[i]));
            }
    }
    auto apply = [&](int act) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int c = 0; c < 8; ++c)
                v[i][c] = activate(act, v[i][c]);
    };
    // one uniform branch on the activation, not one an element
    switch (ACT == kAnyActivation ? e.act : ACT) {
    case GEMM_ACT_RELU: apply(GEMM_ACT_RELU); break;
    case GEMM_ACT_GELU: apply(GEMM_ACT_GELU); break;
    case GEMM_ACT_GELU_TANH: apply(GEMM_ACT_GELU_TANH); break;
    case GEMM_ACT_SILU: apply(GEMM_ACT_SILU); break;
    default: break;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            if (GATED)
                v[i][c] *= u[i][c];
            else if (e.R)
                v[i][c] += r[i][c];
        }
        if (row + i * step < M) {
            const size_t at = (size_t)(row + i * step) * e.ldy + col;
            if (!GATED && e.y_f32)
                store8_f32((float *)e.Y + at, n, v[i]);
            else if (!GATED && e.y_f16)
                store8_16((uint16_t *)e.Y + at, n, pack8<Half16>(v[i]));
            else
                store8_16((uint16_t *)e.Y + at, n, pack8<Fmt>(v[i]));
        }
    }
}

// One row's.
template <class Fmt, bool GATED>
__device__ __forceinline__ void emit8(const Epilogue &e, int row, int col, int n, const float (&v)[8],
                                      const float (&u)[8])
{
    float b[8], v1[1][8], u1[1][8];
    load_bias<Fmt>(e, col, n, b);
#pragma unroll
    for (int c = 0; c < 8; ++c)
        v1[0][c] = v[c], u1[0][c] = u[c];
    emit_rows<Fmt, GATED, false, kAnyActivation, 1>(e, row, 0, row + 1, col, n, v1, u1, b);
}

}  // namespace dgor
