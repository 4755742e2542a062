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

// 1 / (1 + exp(-v)), to a few units of a 32-bit float
__device__ __forceinline__ float logistic(float v) { return rcp_approx(1.0f + exp2_approx(-1.4426950408889634f * v)); }

// The normal distribution function Phi(z) = (1 + erf(z / sqrt 2)) / 2 and exp(-z^2 / 2), by the
// rational approximation of erf in Abramowitz and Stegun, formula 7.1.26 (error below 1.5e-7):
//   1 - erf(a) = (a1 t + .. + a5 t^5) exp(-a^2),  t = 1 / (1 + p a),  a >= 0
// One exponential serves both; erff and expf took about twice the instructions, and the
// backward pass's element-wise kernel was bound by them.
__device__ __forceinline__ float normal_cdf(float z, float& bell)
{
    const float a = fabsf(z) * 0.70710678118654752f;
    const float t = rcp_approx(fmaf(0.3275911f, a, 1.0f));
    bell = exp2_approx(z * z * -0.72134752044448170f);
    float q = fmaf(1.061405429f, t, -1.453152027f);
    q = fmaf(q, t, 1.421413741f);
    q = fmaf(q, t, -0.284496736f);
    q = fmaf(q, t, 0.254829592f);
    const float tail = 0.5f * q * t * bell;
    return z < 0.0f ? tail : 1.0f - tail;
}

// tanh's argument in the approximate GELU, twice (z (1 + tanh u) / 2 = z / (1 + exp(-2u)))
__device__ __forceinline__ float gelu_tanh_argument(float z)
{
    return z * fmaf(0.07135481627260025f, z * z, 1.5957691216057308f);
}

__device__ __forceinline__ float act_value(int act, float z)
{
    switch (act) {
    case ITO_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case ITO_ACT_GELU: {
        float bell;
        return z * normal_cdf(z, bell);
    }
    case ITO_ACT_GELU_TANH: return z * logistic(gelu_tanh_argument(z));
    case ITO_ACT_SILU: return z * logistic(z);
    default: return z;
    }
}

__device__ __forceinline__ float act_slope(int act, float z)
{
    switch (act) {
    case ITO_ACT_RELU: return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
    case ITO_ACT_GELU: {
        float bell;
        const float cdf = normal_cdf(z, bell);
        return fmaf(z * bell, 0.39894228040143268f, cdf);
    }
    case ITO_ACT_GELU_TANH: {
        const float q = logistic(gelu_tanh_argument(z));
        return fmaf(z * fmaf(0.21406444881780075f, z * z, 1.5957691216057308f), q * (1.0f - q), q);
    }
    case ITO_ACT_SILU: {
        const float q = logistic(z);
        return fmaf(z, q * (1.0f - q), q);
    }
    default: return 1.0f;
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
