// Building blocks of the float operators (the float layers, loss and optimizer that train
// beside the integer layers): element types, conversions, vector loads and block sums.
#pragma once

#include <atomic>
#include <type_traits>

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

// 16 bytes of a tensor: kPer elements
template <typename T>
struct Vec {
    static constexpr int kPer = 16 / sizeof(T);
    uint4 raw;

    __device__ __forceinline__ void get(float (&v)[kPer]) const
    {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = lane16(w[i], 0);
                v[2 * i + 1] = lane16(w[i], 1);
            }
        }
    }
    __device__ __forceinline__ void set(const float (&v)[kPer])
    {
        uint32_t w[4];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pair16(v[2 * i], v[2 * i + 1]);
        }
        raw = make_uint4(w[0], w[1], w[2], w[3]);
    }
    // the low or the high half of a word as a 32-bit float, and two of them as a word
    static __device__ __forceinline__ float lane16(uint32_t w, int hi)
    {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(hi ? w & 0xFFFF0000u : w << 16);
        const uint16_t h = hi ? (uint16_t)(w >> 16) : (uint16_t)w;
        return to_f32(*reinterpret_cast<const T*>(&h));
    }
    static __device__ __forceinline__ uint32_t pair16(float lo, float hi)
    {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
            return *reinterpret_cast<const uint32_t*>(&v);
        } else {
            const __half2 v = __floats2half2_rn(lo, hi);
            return *reinterpret_cast<const uint32_t*>(&v);
        }
    }
    // element i, where i differs from lane to lane
    __device__ __forceinline__ float element(int i) const
    {
        const int word = sizeof(T) == 4 ? i : i >> 1;
        const uint32_t lo = word & 1 ? raw.y : raw.x, hi = word & 1 ? raw.w : raw.z;
        const uint32_t w = word & 2 ? hi : lo;
        if constexpr (sizeof(T) == 4) return __uint_as_float(w);
        else return lane16(i & 1 ? w >> 16 : w, 0);
    }
    // the largest element (a NaN counts only where there is nothing else)
    __device__ __forceinline__ float largest() const
    {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        if constexpr (sizeof(T) == 4) {
            return fmaxf(fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1])),
                         fmaxf(__uint_as_float(w[2]), __uint_as_float(w[3])));
        } else {
            const uint32_t m = max_pair(max_pair(w[0], w[1]), max_pair(w[2], w[3]));
            return fmaxf(lane16(m, 0), lane16(m, 1));
        }
    }
    static __device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b)
    {
        uint32_t r;
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
            asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else
            asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    // elements c .. c + kPer - 1 of a row of n, 0 beyond it; vec: the row starts on 16 bytes
    // (c is a multiple of kPer)
    __device__ __forceinline__ void load(const T* row, int c, int n, bool vec)
    {
        if (vec && c + kPer <= n) {
            raw = *reinterpret_cast<const uint4*>(row + c);
            return;
        }
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (c + i < n) {
                if constexpr (sizeof(T) == 4) w[i] = *reinterpret_cast<const uint32_t*>(row + c + i);
                else w[i >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(row + c + i) << (16 * (i & 1));
            }
        raw = make_uint4(w[0], w[1], w[2], w[3]);
    }
    // elements c, c + step, .. of a row of n
    __device__ __forceinline__ void load_apart(const T* row, int c, int step, int n)
    {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (c + i * step < n) {
                if constexpr (sizeof(T) == 4) w[i] = *reinterpret_cast<const uint32_t*>(row + c + i * step);
                else w[i >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(row + c + i * step) << (16 * (i & 1));
            }
        raw = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void store_apart(T* row, int c, int step, int n) const
    {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (c + i * step < n) {
                if constexpr (sizeof(T) == 4) *reinterpret_cast<uint32_t*>(row + c + i * step) = w[i];
                else *reinterpret_cast<uint16_t*>(row + c + i * step) = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            }
    }
    __device__ __forceinline__ void store(T* row, int c, int n, bool vec) const
    {
        if (vec && c + kPer <= n) {
            *reinterpret_cast<uint4*>(row + c) = raw;
            return;
        }
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (c + i < n) {
                if constexpr (sizeof(T) == 4) *reinterpret_cast<uint32_t*>(row + c + i) = w[i];
                else *reinterpret_cast<uint16_t*>(row + c + i) = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            }
    }
};

// rows that 16-byte accesses can take: every row starts on a 16-byte boundary
inline bool rows_vec(const void* p, int64_t ld, size_t size, int64_t rows)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (rows == 1 || ld * (int64_t)size % 16 == 0);
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

// ------------------------------------------------------------------ bulk copies
//
// `bytes` (a multiple of 16) from global to shared memory by the copy engine, both on 16-byte
// boundaries, completing on an mbarrier.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// A place in a ring of `stages` buffers, each with an mbarrier on which its copies complete, and the
// parity of that barrier's phase for the copy at this place.
struct RingPlace {
    int stage;
    uint32_t phase;

    __host__ __device__ __forceinline__ void next(int stages)
    {
        if (++stage < stages) return;
        stage = 0;
        phase ^= 1;
    }
    // One lap back: where a producer whose next copy would go here began its last `stages` copies. (A
    // stage that has had none counts as landed: the phase before a barrier's first is a completed one.)
    __host__ __device__ __forceinline__ RingPlace lap_before() const { return RingPlace{stage, phase ^ 1}; }
};

// Waits, by one thread, until the `copies` copies from `at` on have landed. A block whose waits ran out
// must not leave before: its shared memory would be another's while copies still write to it. All of them
// within the limit of one wait; nothing more can be done for what has not come by then.
inline __device__ __noinline__ void ring_landed(uint64_t* full, int stages, RingPlace at, int copies)
{
    uint64_t t0 = 0;                 // (the timer takes a microsecond: not where copies have landed)
    for (int i = 0; i < copies; ++i, at.next(stages))
        while (!mbar_try_wait(&full[at.stage], at.phase)) {
            const uint64_t t = globaltimer_ns();
            if (!t0) t0 = t;
            if (t - t0 > kWaitTimeoutNs) return;
        }
}

// What has to be done once on each device (a kernel's attributes belong to the function on one device).
// Host threads that meet here may both do it. `call` returns a cudaError_t.
struct OnEachDevice {
    std::atomic<uint64_t> done{0};

    template <typename Call>
    cudaError_t run(int device, Call call)
    {
        const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;     // (0: every time)
        if (done.load() & bit) return cudaSuccess;
        const cudaError_t e = call();
        if (e == cudaSuccess) done.fetch_or(bit);
        return e;
    }
};

inline int launch_status(const char* what)
{
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ITO_OK : set_error(ITO_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

}  // namespace ito
