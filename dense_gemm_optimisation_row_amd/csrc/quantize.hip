// Rows of FP32, binary16 or bfloat16 as 8-bit codes and one FP32 scale each
// (declared in include/gemm.h), the form in which the 8-bit products take their
// operands:
//   scale = max(fl(max |x| fl(1 / 127)), 2^-126),  q = x / scale to the nearest whole
//   number, ties to even.
// q is that of the exact quotient: r = rint(x / scale) in FP32 may be the wrong
// neighbour next to a border, so 2 (x - r scale) is compared with the scale; the
// FMA that gives it is exact, x and r scale being multiples of the scale's last
// place, and their difference at most half the scale.  Any order of the sums gives
// the same, there are none.  A row that holds a NaN or an infinity has no such
// scale: its scale is NaN, its codes are zero.
//
// Bound by memory: a row is held in registers between the maximum and the codes,
// so it is read once.  A row's threads: one wavefront where there are rows for
// all compute units, else 256 or 1024, which have fewer loads after one another.
#include <stdint.h>

#include "common.h"
#include "epilogue.h"
#include "linear.h"

namespace dgor {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_at1 __attribute__((aligned(1)));

struct Rows {
    const void *x;
    int8_t *q;
    float *scale;
    int M, K;
    long long ldx, ldq;
};

// Eight elements as loaded, and what they give.  What is past the row is zero,
// which changes no maximum.
template <class Fmt>
struct Unit {
    static constexpr int BYTES = 2;   // of an element
    u32x4 v;
    __device__ __forceinline__ void load(const void *x, long long at, int n)
    {
        v = n > 0 ? load8_16((const uint16_t *)x + at, n) : u32x4{0u, 0u, 0u, 0u};
    }
    // the largest |x| as its bits in FP32, which are in the values' order
    __device__ __forceinline__ uint32_t top() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t lo = v[e] & 0x7fffu, hi = (v[e] >> 16) & 0x7fffu;
            m = max(m, max(lo, hi));
        }
        return __float_as_uint(Fmt::up((uint16_t)m));
    }
    __device__ __forceinline__ void open(float (&f)[8]) const { unpack8<Fmt>(v, f); }
};
template <>
struct Unit<float> {
    static constexpr int BYTES = 4;
    float v[8];
    __device__ __forceinline__ void load(const void *x, long long at, int n)
    {
        if (n > 0)
            load8_f32((const float *)x + at, n, v);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = 0.f;
    }
    __device__ __forceinline__ uint32_t top() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ void open(float (&f)[8]) const
    {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = v[e];
    }
};

constexpr uint32_t kInfinity = 0x7f800000u;

__device__ __forceinline__ float scale_of(uint32_t top)
{
    const float s = __uint_as_float(top) * (1.f / 127.f);
    return top >= kInfinity ? __uint_as_float(0x7fc00000u) : (s > 0x1p-126f ? s : 0x1p-126f);
}

// The codes of eight elements, n of them inside the row.
template <class Fmt>
__device__ __forceinline__ void put(const Unit<Fmt> &unit, int8_t *q, int n, float scale, float inverse)
{
    float f[8];
    unit.open(f);
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float r = __builtin_rintf(f[e] * inverse);
        const float off = 2.f * __builtin_fmaf(-r, scale, f[e]);
        const int whole = (int)r;
        if (fabsf(off) > scale || (fabsf(off) == scale && (whole & 1)))
            r += __builtin_copysignf(1.f, off);
        b[e] = (uint32_t)(int)r & 0xffu;
    }
    const u32x2 v = {b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24, b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24};
    if (n >= 8) {
        *reinterpret_cast<u32x2_at1 *>(q) = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n)
            q[e] = (int8_t)(v[e >> 2] >> (8 * (e & 3)));
}

// The largest value of a row's threads.
template <int T>
__device__ __forceinline__ uint32_t row_top(uint32_t m, uint32_t *lds)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
    if (T > 64) {
        if ((threadIdx.x & 63) == 0)
            lds[threadIdx.x >> 6] = m;
        __syncthreads();
        m = 0;
#pragma unroll
        for (int w = 0; w < T / 64; ++w)
            m = max(m, lds[w]);
    }
    return m;
}

// T threads a row, U units of eight elements each.
template <class Fmt, int T, int U>
__global__ __launch_bounds__(T > 256 ? T : 256) void quantize_kernel(Rows p)
{
    constexpr int BLOCK = T > 256 ? T : 256;
    __shared__ uint32_t lds[T > 64 ? T / 64 : 1];
    const int row = (int)(blockIdx.x * (BLOCK / T) + threadIdx.x / T), t = (int)(threadIdx.x % T);
    if (row >= p.M)
        return;   // whole wavefronts, and with them every thread of the row
    Unit<Fmt> u[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int c = 8 * (t + T * i);
        u[i].load(p.x, row * p.ldx + c, p.K - c);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < U; ++i)
        m = max(m, u[i].top());
    const float s = scale_of(row_top<T>(m, lds));
    if (t == 0)
        p.scale[row] = s;
    const bool none = s != s;
    const float held = none ? 1.f : s, inverse = none ? 0.f : __builtin_amdgcn_rcpf(s);
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int c = 8 * (t + T * i);
        if (none)
            u[i] = Unit<Fmt>{};
        if (c < p.K)
            put(u[i], p.q + row * p.ldq + c, p.K - c, held, inverse);
    }
}

// Rows longer than the registers of 1024 threads hold: read twice.
template <class Fmt>
__global__ __launch_bounds__(1024) void quantize_long_kernel(Rows p)
{
    __shared__ uint32_t lds[16];
    const long long row = blockIdx.x;
    uint32_t m = 0;
    for (long long c = 8 * threadIdx.x; c < p.K; c += 8 * 1024) {
        Unit<Fmt> u;
        u.load(p.x, row * p.ldx + c, (int)(p.K - c));
        m = max(m, u.top());
    }
    const float s = scale_of(row_top<1024>(m, lds));
    if (threadIdx.x == 0)
        p.scale[row] = s;
    const bool none = s != s;
    const float held = none ? 1.f : s, inverse = none ? 0.f : __builtin_amdgcn_rcpf(s);
    for (long long c = 8 * threadIdx.x; c < p.K; c += 8 * 1024) {
        Unit<Fmt> u;
        u.load(p.x, row * p.ldx + c, (int)(p.K - c));
        if (none)
            u = Unit<Fmt>{};
        put(u, p.q + row * p.ldq + c, (int)(p.K - c), held, inverse);
    }
}

template <class Fmt, int T>
hipError_t launch_rows(const Rows &p, hipStream_t s)
{
    constexpr int BLOCK = T > 256 ? T : 256, ROWS = BLOCK / T;
    const dim3 grid((unsigned)((p.M + ROWS - 1LL) / ROWS)), block(BLOCK);
    const int units = (p.K + 8 * T - 1) / (8 * T);
    if (units <= 1)
        hipLaunchKernelGGL((quantize_kernel<Fmt, T, 1>), grid, block, 0, s, p);
    else if (units <= 2)
        hipLaunchKernelGGL((quantize_kernel<Fmt, T, 2>), grid, block, 0, s, p);
    else if (units <= 4)
        hipLaunchKernelGGL((quantize_kernel<Fmt, T, 4>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((quantize_kernel<Fmt, T, 8>), grid, block, 0, s, p);
    return hipGetLastError();
}

template <class Fmt>
hipError_t launch(const Rows &p, hipStream_t s)
{
    if (p.K <= 64 * 64 && (p.M >= 1024 || p.K <= 512))
        return launch_rows<Fmt, 64>(p, s);
    if (p.K <= 256 * 64)
        return launch_rows<Fmt, 256>(p, s);
    if (p.K <= 1024 * 64)
        return launch_rows<Fmt, 1024>(p, s);
    hipLaunchKernelGGL((quantize_long_kernel<Fmt>), dim3((unsigned)p.M), dim3(1024), 0, s, p);
    return hipGetLastError();
}

template <class Fmt>
int run(const gemm_quantize_i8_params *q, const void *x, int8_t *codes, float *scale, void *stream)
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    if (q->M < 0 || q->K < 0 || q->K > 0x7fffffff - 65536)
        return GEMM_ERR_INVALID_DIM;
    if (q->ldx < (q->K > 1 ? q->K : 1) || q->ldq < (q->K > 1 ? q->K : 1))
        return GEMM_ERR_INVALID_LAYOUT;
    if (q->M > 0 && ((q->K > 0 && (!x || !codes)) || !scale))
        return GEMM_ERR_NULL_PTR;
    if (q->M == 0)
        return GEMM_OK;
    const int dev = device_status();
    if (dev != GEMM_OK)
        return dev;
    // a launch holds fewer than 2^32 threads, of which a row has up to 1024
    constexpr int MOST = 1 << 21;
    for (long long r = 0; r < q->M; r += MOST) {
        const Rows p{(const char *)x + r * q->ldx * Unit<Fmt>::BYTES, codes + r * q->ldq, scale + r,
                     (int)(q->M - r < MOST ? q->M - r : MOST), q->K, q->ldx, q->ldq};
        if (launch<Fmt>(p, (hipStream_t)stream) != hipSuccess)
            return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

}  // namespace
}  // namespace dgor

extern "C" {

int gemm_quantize_i8_f32(const gemm_quantize_i8_params *params, const float *x, int8_t *q, float *scale, void *stream)
{
    return dgor::run<float>(params, x, q, scale, stream);
}
int gemm_quantize_i8_f16(const gemm_quantize_i8_params *params, const uint16_t *x, int8_t *q, float *scale,
                         void *stream)
{
    return dgor::run<dgor::Half16>(params, x, q, scale, stream);
}
int gemm_quantize_i8_bf16(const gemm_quantize_i8_params *params, const uint16_t *x, int8_t *q, float *scale,
                          void *stream)
{
    return dgor::run<dgor::Brain16>(params, x, q, scale, stream);
}

}  // extern "C"
