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

// exp and 1 / (1 + e) of a gate.  Rows of 16 bits take the hardware's exp2 directly (2^-22 relative and
// 2^-24 |x log2 e| from rounding its argument): z itself was rounded by 2^-9 |z| (bf16) or 2^-12 |z| (fp16),
// so its coefficient is already uncertain by over 100 times that, and the exact function's extra
// instructions would show at one pass over memory.  The hardware's reciprocal is 2^-23 relative.
template <bool FAST>
__device__ __forceinline__ float gate_exp(float x)
{
    if constexpr (FAST) {
        float r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
        return r;
    } else
        return expf(x);
}
template <bool FAST>
__device__ __forceinline__ double gate_exp(double x) { return exp(x); }
__device__ __forceinline__ float gate_rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ double gate_rcp(double x) { return 1.0 / x; }

// Coefficient a and input weight w of a stored gate value z.  Both halves of the sigmoid come from
// one e = exp(-z), a = 1 / (1 + e) and w = e a, so that 1 - a keeps its digits where a rounds to 1.  z
// is held above -86 (fp64: -700), where e would leave the range and a is below 1e-37 anyway.
template <int GATE, bool FAST, typename A>
__device__ __forceinline__ void gate_of(A z, A &a, A &w)
{
    if constexpr (GATE == SLA_GATE_VALUE) {
        a = z;
        w = A(1);
    } else if constexpr (GATE == SLA_GATE_EXP) {
        a = gate_exp<FAST>(z);
        w = A(1);
    } else {
        const A floor = sizeof(A) == 4 ? A(-86) : A(-700);
        const A e = gate_exp<FAST>(-(z < floor ? floor : z));   // a NaN stays one
        a = gate_rcp(A(1) + e);
        w = e * a;
    }
}

}  // namespace sla
