// Building blocks of the float operators (the float layers, loss and optimizer that train
// beside the integer layers): element types, conversions, vector loads and block sums.
#pragma once

#include <cuda_fp16.h>

#include "ito_device.cuh"
#include "ito_internal.h"

namespace ito {

// ---------------------------------------------------------------- element types

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

// rounded to nearest, ties to even (the one rounding of a result to its type)
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// element i of a tensor whose type is known at run time only (small vectors: biases, norms' weights)
__device__ __forceinline__ float load_typed(const void* p, int type, int64_t i)
{
    if (type == ITO_F32) return static_cast<const float*>(p)[i];
    if (type == ITO_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}

inline size_t type_bytes(int type) { return type == ITO_F32 ? 4 : 2; }
inline bool type_known(int type) { return type == ITO_F32 || type == ITO_BF16 || type == ITO_F16; }
inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// ------------------------------------------------------------------- reductions

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

inline int launch_status(const char* what)
{
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ITO_OK : set_error(ITO_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

}  // namespace ito
