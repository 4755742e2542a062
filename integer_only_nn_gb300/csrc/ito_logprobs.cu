// Log probabilities of given tokens (class labels), with the distribution's entropy and its
// largest alternatives, and the gradient of the first two.
//
//   top = max x    s = sum exp(x - top)    lse = top + log s
//   logp = x[target] - lse                 H = log s - (sum (x - top) exp(x - top)) / s
//   dx_j = g_logp (hot_j - p_j) - g_H p_j (log p_j + H),      p = exp(x - lse)
//
// Masked classes hold -inf: they have p = 0 and take no part. A row whose every class is
// masked has lse = -inf, log probabilities of -inf, entropy 0 and a gradient of 0. A target
// of -1 stands for no token: logp 0 and no gradient from it.
#include <climits>
#include <cmath>

#include "ito_float.cuh"

namespace ito {

constexpr int kLpThreads = 256;
constexpr int kLpMaxTop = 32;

// larger values first, equal values in the order of their index; a NaN above all
__device__ __forceinline__ bool comes_before(float a, int ia, float b, int ib)
{
    if (a > b) return true;
    if (a < b) return false;
    const bool na = a != a, nb = b != b;
    if (na != nb) return na;
    return ia < ib;
}

// the sums of a part of a row: its largest value, sum exp(x - top), sum (x - top) exp(x - top)
struct Sums {
    float top, s, t;
};

__device__ __forceinline__ Sums join(const Sums& a, const Sums& b)
{
    if (b.s == 0.0f) return a;
    if (a.s == 0.0f) return b;
    const float top = fmaxf(a.top, b.top);
    const float ea = expf(a.top - top), eb = expf(b.top - top);
    return Sums{top, a.s * ea + b.s * eb, (a.t + (a.top - top) * a.s) * ea + (b.t + (b.top - top) * b.s) * eb};
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads)
    k_logprobs_fwd(const T* __restrict__ x, int64_t ld, const int32_t* __restrict__ targets, int64_t rows, int classes,
                   int k, float* __restrict__ logp, float* __restrict__ entropy, float* __restrict__ lse,
                   int32_t* __restrict__ top_ids, float* __restrict__ top_logp, int* __restrict__ err)
{
    griddep_wait();
    griddep_launch_dependents();
    __shared__ Sums part[kLpThreads];
    __shared__ float bv[kLpThreads];
    __shared__ int bi[kLpThreads];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* xr = x + r * ld;
        Sums a{0.0f, 0.0f, 0.0f};
        float top = -INFINITY;
        for (int c = threadIdx.x; c < classes; c += kLpThreads) {
            const float v = to_f32(xr[c]);
            top = v > top || v != v ? v : top;
        }
        bv[threadIdx.x] = top;
        __syncthreads();
        for (int o = kLpThreads / 2; o > 0; o >>= 1) {
            if (threadIdx.x < o) {
                const float b = bv[threadIdx.x + o];
                if (b > bv[threadIdx.x] || b != b) bv[threadIdx.x] = b;
            }
            __syncthreads();
        }
        top = bv[0];
        a.top = top;
        for (int c = threadIdx.x; c < classes; c += kLpThreads) {
            const float v = to_f32(xr[c]);
            if (v == -INFINITY) continue;
            const float e = expf(v - top);
            a.s += e;
            a.t += e != 0.0f ? (v - top) * e : 0.0f;
        }
        part[threadIdx.x] = a;
        __syncthreads();
        for (int o = kLpThreads / 2; o > 0; o >>= 1) {
            if (threadIdx.x < o) part[threadIdx.x] = join(part[threadIdx.x], part[threadIdx.x + o]);
            __syncthreads();
        }
        a = part[0];
        const float ls = logf(a.s);
        const bool none = a.s == 0.0f;
        const float z = none ? -INFINITY : a.top + ls;
        if (threadIdx.x == 0) {
            if (lse) lse[r] = z;
            if (entropy) entropy[r] = none ? 0.0f : ls - a.t / a.s;
            if (logp) {
                const int t = targets[r];
                if (t < -1 || t >= classes) raise_device_error(err, ITO_ERR_ARG);
                logp[r] = t < 0 || t >= classes ? 0.0f : none ? -INFINITY : to_f32(xr[t]) - z;
            }
        }
        float last = 0.0f;
        int last_i = -1;
        for (int j = 0; j < k; ++j) {
            float best = -INFINITY;
            int best_i = INT_MAX;
            for (int c = threadIdx.x; c < classes; c += kLpThreads) {
                const float v = to_f32(xr[c]);
                if (j && !comes_before(last, last_i, v, c)) continue;
                if (comes_before(v, c, best, best_i)) { best = v; best_i = c; }
            }
            __syncthreads();
            bv[threadIdx.x] = best;
            bi[threadIdx.x] = best_i;
            __syncthreads();
            for (int o = kLpThreads / 2; o > 0; o >>= 1) {
                if (threadIdx.x < o && comes_before(bv[threadIdx.x + o], bi[threadIdx.x + o], bv[threadIdx.x], bi[threadIdx.x])) {
                    bv[threadIdx.x] = bv[threadIdx.x + o];
                    bi[threadIdx.x] = bi[threadIdx.x + o];
                }
                __syncthreads();
            }
            last = bv[0];
            last_i = bi[0];
            if (threadIdx.x == 0) {
                top_ids[r * k + j] = last_i;
                top_logp[r * k + j] = none ? -INFINITY : last - z;
            }
        }
        __syncthreads();
    }
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads)
    k_logprobs_bwd(const T* __restrict__ x, int64_t ld, const int32_t* __restrict__ targets,
                   const float* __restrict__ lse, const float* __restrict__ entropy, int64_t rows, int classes,
                   const float* __restrict__ g_logp, const float* __restrict__ g_entropy, T* __restrict__ dx,
                   int64_t ldd, int* __restrict__ err)
{
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const float z = lse[r];
        int t = targets ? targets[r] : -1;
        if (t < -1 || t >= classes) {
            if (threadIdx.x == 0) raise_device_error(err, ITO_ERR_ARG);
            t = -1;
        }
        const float g = t >= 0 && g_logp ? g_logp[r] : 0.0f;
        const float gh = g_entropy ? g_entropy[r] : 0.0f, h = g_entropy ? entropy[r] : 0.0f;
        for (int c = threadIdx.x; c < classes; c += kLpThreads) {
            const float v = to_f32(x[r * ld + c]);
            float d = 0.0f;
            if (z != -INFINITY) {
                const float lp = v - z;
                d = c == t ? g : 0.0f;
                if (v != -INFINITY) d -= expf(lp) * (g + gh * (lp + h));
            }
            dx[r * ldd + c] = from_f32<T>(d);
        }
    }
}

static int check_lp(const void* x, int64_t ld, int type, int64_t rows, int classes)
{
    if (!x) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    if (!type_known(type)) return set_error(ITO_ERR_ARG, "unknown type");
    if (rows < 1 || classes < 1) return set_error(ITO_ERR_SHAPE, "sizes must be >= 1");
    if (rows > (int64_t(1) << 40) || classes > (1 << 30)) return set_error(ITO_ERR_SHAPE, "rows above 2^40 or classes above 2^30");
    if (rows > 1 && ld < classes) return set_error(ITO_ERR_SHAPE, "row stride below classes");
    if (!aligned_to(x, type_bytes(type))) return set_error(ITO_ERR_ARG, "misaligned pointer");
    return ITO_OK;
}

template <typename T>
static int run_fwd(const void* x, int64_t ld, const int32_t* targets, int64_t rows, int classes, int k, float* logp,
                   float* entropy, float* lse, int32_t* top_ids, float* top_logp, int* err, cudaStream_t s)
{
    const int64_t grid = rows < 8 * num_sms() ? rows : 8 * num_sms();
    launch_pdl(k_logprobs_fwd<T>, (unsigned)grid, kLpThreads, 0, s, static_cast<const T*>(x), ld, targets, rows,
               classes, k, logp, entropy, lse, top_ids, top_logp, err);
    return launch_status("log probabilities");
}

template <typename T>
static int run_bwd(const void* x, int64_t ld, const int32_t* targets, const float* lse, const float* entropy,
                   int64_t rows, int classes, const float* g_logp, const float* g_entropy, void* dx, int64_t ldd,
                   int* err, cudaStream_t s)
{
    const int64_t grid = rows < 8 * num_sms() ? rows : 8 * num_sms();
    launch_pdl(k_logprobs_bwd<T>, (unsigned)grid, kLpThreads, 0, s, static_cast<const T*>(x), ld, targets, lse,
               entropy, rows, classes, g_logp, g_entropy, static_cast<T*>(dx), ldd, err);
    return launch_status("log probabilities");
}

}  // namespace ito

using namespace ito;

extern "C" {

int ito_token_logprobs_fwd(const void* logits, int64_t ld, int type, const int32_t* targets, int64_t rows, int classes,
                           int k, float* logp, float* entropy, float* lse, int32_t* top_ids, float* top_logp,
                           void* stream)
{
    const int r = check_lp(logits, ld, type, rows, classes);
    if (r) return r;
    if (k < 0 || k > kLpMaxTop) return set_error(ITO_ERR_ARG, "k must be in 0 .. %d", kLpMaxTop);
    if (k > classes) return set_error(ITO_ERR_SHAPE, "k above classes");
    if (k && (!top_ids || !top_logp)) return set_error(ITO_ERR_ARG, "NULL top_ids or top_logp");
    if (logp && !targets) return set_error(ITO_ERR_ARG, "logp needs targets");
    if (!k && !logp && !entropy && !lse) return set_error(ITO_ERR_ARG, "no output");
    if (!aligned_to(targets, 4) || !aligned_to(logp, 4) || !aligned_to(entropy, 4) || !aligned_to(lse, 4) ||
        !aligned_to(top_ids, 4) || !aligned_to(top_logp, 4))
        return set_error(ITO_ERR_ARG, "misaligned pointer");
    int* err = device_error_word();
    if (!err) return set_error(ITO_ERR_CUDA, "device error word unavailable");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (type == ITO_F32)
        return run_fwd<float>(logits, ld, targets, rows, classes, k, logp, entropy, lse, top_ids, top_logp, err, s);
    if (type == ITO_BF16)
        return run_fwd<__nv_bfloat16>(logits, ld, targets, rows, classes, k, logp, entropy, lse, top_ids, top_logp,
                                      err, s);
    return run_fwd<__half>(logits, ld, targets, rows, classes, k, logp, entropy, lse, top_ids, top_logp, err, s);
}

int ito_token_logprobs_bwd(const void* logits, int64_t ld, int type, const int32_t* targets, const float* lse,
                           const float* entropy, int64_t rows, int classes, const float* g_logp,
                           const float* g_entropy, void* dlogits, int64_t ldd, void* stream)
{
    const int r = check_lp(logits, ld, type, rows, classes);
    if (r) return r;
    if (!lse || !dlogits || (!g_logp && !g_entropy)) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    if (g_logp && !targets) return set_error(ITO_ERR_ARG, "g_logp needs targets");
    if (g_entropy && !entropy) return set_error(ITO_ERR_ARG, "g_entropy needs entropy");
    if (rows > 1 && ldd < classes) return set_error(ITO_ERR_SHAPE, "row stride below classes");
    if (!aligned_to(dlogits, type_bytes(type)) || !aligned_to(targets, 4) || !aligned_to(lse, 4) ||
        !aligned_to(entropy, 4) || !aligned_to(g_logp, 4) || !aligned_to(g_entropy, 4))
        return set_error(ITO_ERR_ARG, "misaligned pointer");
    int* err = device_error_word();
    if (!err) return set_error(ITO_ERR_CUDA, "device error word unavailable");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (type == ITO_F32)
        return run_bwd<float>(logits, ld, targets, lse, entropy, rows, classes, g_logp, g_entropy, dlogits, ldd, err, s);
    if (type == ITO_BF16)
        return run_bwd<__nv_bfloat16>(logits, ld, targets, lse, entropy, rows, classes, g_logp, g_entropy, dlogits,
                                      ldd, err, s);
    return run_bwd<__half>(logits, ld, targets, lse, entropy, rows, classes, g_logp, g_entropy, dlogits, ldd, err, s);
}

}  // extern "C"
