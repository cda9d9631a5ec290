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

// exp and 1 / (1 + e) of a gate, e in [0, 1].  Rows of 16 bits take the hardware's exp2 and reciprocal
// (__expf: (2 + 1.2 |x|) 2^-23 relative): z itself was rounded to 2^-9 |z| (bf16) or 2^-12 |z| (fp16), so
// its coefficient is already uncertain by over 100 times that, and the exact functions' extra
// instructions would show at one pass over memory.
template <bool FAST>
__device__ __forceinline__ float gate_exp(float x) { return FAST ? __expf(x) : expf(x); }
template <bool FAST>
__device__ __forceinline__ double gate_exp(double x) { return exp(x); }
template <bool FAST>
__device__ __forceinline__ float gate_rcp(float x) { return FAST ? __fdividef(1.0f, x) : __frcp_rn(x); }
template <bool FAST>
__device__ __forceinline__ double gate_rcp(double x) { return 1.0 / x; }

// Coefficient a and input weight w of a stored gate value z.  The sigmoid's two halves come from
// one e = exp(-|z|): 1/(1+e) and e/(1+e), so that 1 - a keeps its digits where a rounds to 1.
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
        const A e = gate_exp<FAST>(z < A(0) ? z : -z);
        const A big = gate_rcp<FAST>(A(1) + e), small = e * big;
        a = z < A(0) ? small : big;
        w = z < A(0) ? big : small;
    }
}

}  // namespace sla
