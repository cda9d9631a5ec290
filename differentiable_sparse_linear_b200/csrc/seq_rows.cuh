// Row types of the sequence operators (recur.cu, route.cu): storage type -> arithmetic type, and
// the gates of the recurrence.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "sla.h"
#include "sla_internal.cuh"

namespace sla {

// Storage type S and the type A its values are computed in: fp32 for 16- and 32-bit storage, so
// that each value is rounded to its storage type once, when it is written.
template <typename S>
struct RowType;
template <>
struct RowType<float> {
    using A = float;
    static __device__ __forceinline__ float up(float v) { return v; }
    static __device__ __forceinline__ float down(float v) { return v; }
};
template <>
struct RowType<double> {
    using A = double;
    static __device__ __forceinline__ double up(double v) { return v; }
    static __device__ __forceinline__ double down(double v) { return v; }
};
template <>
struct RowType<__nv_bfloat16> {
    using A = float;
    static __device__ __forceinline__ float up(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 down(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct RowType<__half> {
    using A = float;
    static __device__ __forceinline__ float up(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half down(float v) { return __float2half_rn(v); }
};

// f(tag) with tag a value of the storage type of `dtype` (already checked by row_dtype_ok).
template <class F>
static inline sla_status with_row_type(int32_t dtype, F f)
{
    switch (dtype) {
    case SLA_F32: return f(float());
    case SLA_F64: return f(double());
    case SLA_BF16: return f(__nv_bfloat16());
    default: return f(__half());
    }
}

static inline bool row_dtype_ok(int32_t dtype) { return dtype >= SLA_F32 && dtype <= SLA_F16; }
static inline size_t row_bytes(int32_t dtype) { return dtype == SLA_F64 ? 8 : dtype == SLA_F32 ? 4 : 2; }

// SMs of the current device (recur.cu)
int sm_count();

// sums and products that are never contracted, so that every variant of a loop rounds alike
__device__ __forceinline__ float add_of(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ double add_of(double a, double b) { return __dadd_rn(a, b); }
__device__ __forceinline__ float mul_of(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ double mul_of(double a, double b) { return __dmul_rn(a, b); }
__device__ __forceinline__ float fma_of(float a, float b, float c) { return __fmaf_rn(a, b, c); }
__device__ __forceinline__ double fma_of(double a, double b, double c) { return __fma_rn(a, b, c); }

// 16 bytes of a row <-> arithmetic values.
__device__ __forceinline__ void unpack16(const uint4 &r, float (&x)[4], float)
{
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack16(const uint4 &r, double (&x)[2], double)
{
    x[0] = __hiloint2double((int)r.y, (int)r.x);
    x[1] = __hiloint2double((int)r.w, (int)r.z);
}
__device__ __forceinline__ void unpack16(const uint4 &r, float (&x)[8], __nv_bfloat16)
{
    const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack16(const uint4 &r, float (&x)[8], __half)
{
    const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ uint4 pack16(const float (&x)[4], float)
{
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}
__device__ __forceinline__ uint4 pack16(const double (&x)[2], double)
{
    return make_uint4((unsigned)__double2loint(x[0]), (unsigned)__double2hiint(x[0]), (unsigned)__double2loint(x[1]),
                      (unsigned)__double2hiint(x[1]));
}
__device__ __forceinline__ uint4 pack16(const float (&x)[8], __nv_bfloat16)
{
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const unsigned *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack16(const float (&x)[8], __half)
{
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 p = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const unsigned *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Arithmetic on a thread's N values; fp32 in pairs, one instruction for two (rounded as the single ones).
template <int N>
__device__ __forceinline__ void vfma(float (&d)[N], const float (&a)[N], const float (&b)[N], const float (&c)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 2)
        asm("{ .reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
            "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d; }"
            : "=f"(d[i]), "=f"(d[i + 1])
            : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]), "f"(c[i]), "f"(c[i + 1]));
}
template <int N>
__device__ __forceinline__ void vmul(float (&d)[N], const float (&a)[N], const float (&b)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 2)
        asm("{ .reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\t"
            "mov.b64 {%0, %1}, d; }"
            : "=f"(d[i]), "=f"(d[i + 1])
            : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]));
}
template <int N>
__device__ __forceinline__ void vadd(float (&d)[N], const float (&a)[N], const float (&b)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 2)
        asm("{ .reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\t"
            "mov.b64 {%0, %1}, d; }"
            : "=f"(d[i]), "=f"(d[i + 1])
            : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]));
}
template <int N>
__device__ __forceinline__ void vfma(double (&d)[N], const double (&a)[N], const double (&b)[N], const double (&c)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        d[i] = __fma_rn(a[i], b[i], c[i]);
}
template <int N>
__device__ __forceinline__ void vmul(double (&d)[N], const double (&a)[N], const double (&b)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        d[i] = __dmul_rn(a[i], b[i]);
}
template <int N>
__device__ __forceinline__ void vadd(double (&d)[N], const double (&a)[N], const double (&b)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        d[i] = __dadd_rn(a[i], b[i]);
}
template <typename A, int N>
__device__ __forceinline__ void vset(A (&d)[N], A x)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        d[i] = x;
}

__device__ __forceinline__ float ex2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// the hardware's reciprocal, 2^-23 relative
__device__ __forceinline__ float rcp_of(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ double rcp_of(double x) { return 1.0 / x; }

// Coefficients a and input weights w of stored gate values z.
//
// exp: rows of 16 bits take the hardware's exp2 (2^-22 relative), except near 0, where a coefficient near 1 carries
// a state over 1 / |z| rows and its error counts as often: there 1 + z (1 + z/2 + ... + z^5/720), whose
// truncation at |z| = 1/4 is 2^-26 and whose error is the rounding of the last sum.
//
// sigmoid: both halves come from one e = exp(-z), a = 1 / (1 + e) and w = e a, so that 1 - a keeps its digits where
// a rounds to 1, and the larger a is 1 - w, rounded once: the approximate reciprocal's errors have one sign, and a
// state carried over ten thousand rows collected them (2700 units of 2^-24, 620 so).  z is held above -86 (fp64: -700),
// where e would leave the range and a is below 1e-37 anyway.  An error of e counts 1 - a times in a, so the plain
// exp2 is enough for 16-bit rows.
template <int GATE, bool FAST, typename A, int N>
__device__ __forceinline__ void gates_of(const A (&z)[N], A (&a)[N], A (&w)[N])
{
    if constexpr (GATE == SLA_GATE_VALUE) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            a[i] = z[i];
        vset(w, A(1));
    } else if constexpr (GATE == SLA_GATE_EXP) {
        vset(w, A(1));
        if constexpr (FAST) {
            float t[N], q[N], c[N];
            vset(c, 1.4426950408889634f);
            vmul(t, z, c);
            vset(q, 1.0f / 720.0f);
            vset(c, 1.0f / 120.0f);
            vfma(q, z, q, c);
            vset(c, 1.0f / 24.0f);
            vfma(q, z, q, c);
            vset(c, 1.0f / 6.0f);
            vfma(q, z, q, c);
            vset(c, 0.5f);
            vfma(q, z, q, c);
            vset(c, 1.0f);
            vfma(q, z, q, c);
            vfma(q, z, q, c);
#pragma unroll
            for (int i = 0; i < N; ++i)
                a[i] = fabsf(z[i]) < 0.25f ? q[i] : ex2_approx(t[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                a[i] = exp(z[i]);
        }
    } else {
        A e[N];
        if constexpr (FAST) {
            float c[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                e[i] = z[i] < -86.0f ? -86.0f : z[i];      // a NaN stays one
            vset(c, -1.4426950408889634f);
            vmul(e, e, c);
#pragma unroll
            for (int i = 0; i < N; ++i)
                e[i] = ex2_approx(e[i]);
        } else {
            const A floor = sizeof(A) == 4 ? A(-86) : A(-700);
#pragma unroll
            for (int i = 0; i < N; ++i)
                e[i] = exp(-(z[i] < floor ? floor : z[i]));
        }
        vset(a, A(1));
        vadd(a, a, e);
#pragma unroll
        for (int i = 0; i < N; ++i)
            a[i] = rcp_of(a[i]);
        vmul(w, e, a);
#pragma unroll
        for (int i = 0; i < N; ++i)
            a[i] = a[i] <= w[i] ? a[i] : add_of(A(1), -w[i]);
    }
}

}  // namespace sla
