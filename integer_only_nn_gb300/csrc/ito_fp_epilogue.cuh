// Activations and the element-wise end of the linear layer's products.
#pragma once

#include "ito_float.cuh"
#include "ito_fp.h"

namespace ito {

__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

// Activations and their slopes are computed for two elements at a time with packed operations:
// one at a time they bound the backward pass's element-wise kernel (30 instructions an element,
// most of them the GELU's).

// 1 / (1 + exp(-v)), to a few units of a 32-bit float
__device__ __forceinline__ float2 logistic(float2 v)
{
    const float2 y = __fmul2_rn(v, splat(-1.4426950408889634f));
    const float2 d = __fadd2_rn(make_float2(exp2_approx(y.x), exp2_approx(y.y)), splat(1.0f));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}

// The normal distribution function Phi(z) = (1 + erf(z / sqrt 2)) / 2 and exp(-z^2 / 2), by the
// rational approximation of erf in Abramowitz and Stegun, formula 7.1.26 (error below 1.5e-7):
//   1 - erf(a) = (a1 t + .. + a5 t^5) exp(-a^2),  t = 1 / (1 + p a),  a = |z| / sqrt 2
// (the coefficients below are halved, p divided by sqrt 2). One exponential serves both.
__device__ __forceinline__ float2 normal_cdf(float2 z, float2& bell)
{
    const float2 d = __ffma2_rn(make_float2(fabsf(z.x), fabsf(z.y)), splat(0.23164189f), splat(1.0f));
    const float2 t = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    const float2 y = __fmul2_rn(__fmul2_rn(z, z), splat(-0.72134752044448170f));
    bell = make_float2(exp2_approx(y.x), exp2_approx(y.y));
    float2 q = __ffma2_rn(splat(0.5307027145f), t, splat(-0.7265760135f));
    q = __ffma2_rn(q, t, splat(0.7107068705f));
    q = __ffma2_rn(q, t, splat(-0.142248368f));
    q = __ffma2_rn(q, t, splat(0.127414796f));
    const float2 tail = __fmul2_rn(__fmul2_rn(q, t), bell);
    const float2 rest = __ffma2_rn(tail, splat(-1.0f), splat(1.0f));
    return make_float2(z.x < 0.0f ? tail.x : rest.x, z.y < 0.0f ? tail.y : rest.y);
}

// twice tanh's argument in the approximate GELU (z (1 + tanh u) / 2 = z / (1 + exp(-2u))), over z
__device__ __forceinline__ float2 gelu_tanh_factor(float2 z2)
{
    return __ffma2_rn(z2, splat(0.07135481627260025f), splat(1.5957691216057308f));
}

template <int ACT>
__device__ __forceinline__ float2 act_value(float2 z)
{
    if (ACT == ITO_ACT_RELU) return make_float2(z.x < 0.0f ? 0.0f : z.x, z.y < 0.0f ? 0.0f : z.y);
    if (ACT == ITO_ACT_GELU) {
        float2 bell;
        return __fmul2_rn(z, normal_cdf(z, bell));
    }
    if (ACT == ITO_ACT_GELU_TANH) return __fmul2_rn(z, logistic(__fmul2_rn(z, gelu_tanh_factor(__fmul2_rn(z, z)))));
    if (ACT == ITO_ACT_SILU) return __fmul2_rn(z, logistic(z));
    return z;
}

template <int ACT>
__device__ __forceinline__ float2 act_slope(float2 z)
{
    if (ACT == ITO_ACT_RELU)
        return make_float2(z.x > 0.0f ? 1.0f : z.x <= 0.0f ? 0.0f : z.x, z.y > 0.0f ? 1.0f : z.y <= 0.0f ? 0.0f : z.y);
    if (ACT == ITO_ACT_GELU) {
        float2 bell;
        const float2 cdf = normal_cdf(z, bell);
        return __ffma2_rn(__fmul2_rn(z, bell), splat(0.39894228040143268f), cdf);
    }
    if (ACT == ITO_ACT_GELU_TANH || ACT == ITO_ACT_SILU) {
        // q + z u' q (1 - q) with q = logistic(u). From |z| = 11 on q (1 - q) is 0 in the approximate
        // GELU, and z u' is taken at +-16 at most: a cube, it would be infinite from 1e13 on.
        const float2 z2 = __fmul2_rn(z, z);
        const bool silu = ACT == ITO_ACT_SILU;
        const float2 q = logistic(silu ? z : __fmul2_rn(z, gelu_tanh_factor(z2)));
        float2 zu = z;
        if (!silu) {
            const float2 c = make_float2(fminf(fmaxf(z.x, -16.0f), 16.0f), fminf(fmaxf(z.y, -16.0f), 16.0f));
            zu = __fmul2_rn(c, __ffma2_rn(__fmul2_rn(c, c), splat(0.21406444881780075f), splat(1.5957691216057308f)));
        }
        return __ffma2_rn(zu, __fmul2_rn(q, __ffma2_rn(q, splat(-1.0f), splat(1.0f))), q);
    }
    return splat(1.0f);
}

// an activation that is known at run time only
__device__ __forceinline__ float act_value(int act, float z)
{
    switch (act) {
    case ITO_ACT_RELU: return act_value<ITO_ACT_RELU>(splat(z)).x;
    case ITO_ACT_GELU: return act_value<ITO_ACT_GELU>(splat(z)).x;
    case ITO_ACT_GELU_TANH: return act_value<ITO_ACT_GELU_TANH>(splat(z)).x;
    case ITO_ACT_SILU: return act_value<ITO_ACT_SILU>(splat(z)).x;
    default: return z;
    }
}

__device__ __forceinline__ void store_typed(void* p, int type, int64_t i, float v)
{
    if (type == ITO_F32) static_cast<float*>(p)[i] = v;
    else if (type == ITO_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// one element's epilogue
__device__ __forceinline__ void fp_finish(const FpEpilogue& e, int64_t r, int64_t c, float v)
{
    if (e.bias) v += load_typed(e.bias, e.bias_type, c);
    if (e.z) store_typed(e.z, e.type, r * e.ldz + c, v);
    v = act_value(e.act, v);
    if (e.residual) v += load_typed(e.residual, e.out_type, r * e.ldr + c);
    store_typed(e.y, e.out_type, r * e.ldy + c, v);
}

// two floats as one word of two 16-bit floats, lo in the low half
__device__ __forceinline__ uint32_t pack16(int type, float lo, float hi)
{
    if (type == ITO_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float2 unpack16(int type, uint32_t w)
{
    if (type == ITO_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

}  // namespace ito
