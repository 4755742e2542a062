// Activations and the element-wise end of the linear layer's products.
#pragma once

#include "ito_float.cuh"
#include "ito_fp.h"

namespace ito {

__device__ __forceinline__ float act_value(int act, float z)
{
    switch (act) {
    case ITO_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case ITO_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case ITO_ACT_GELU_TANH: return 0.5f * z * (1.0f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
    case ITO_ACT_SILU: return z / (1.0f + expf(-z));
    default: return z;
    }
}

__device__ __forceinline__ float act_slope(int act, float z)
{
    switch (act) {
    case ITO_ACT_RELU: return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
    case ITO_ACT_GELU:
        return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
    case ITO_ACT_GELU_TANH: {
        const float t = tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z));
        return 0.5f * (1.0f + t) + 0.5f * z * (1.0f - t * t) * (0.79788456080286536f * (1.0f + 0.134145f * z * z));
    }
    case ITO_ACT_SILU: {
        const float q = 1.0f / (1.0f + expf(-z));
        return q * (1.0f + z * (1.0f - q));
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
