// Linear layer on 16-bit floats with its epilogue fused, and its backward pass.
//
//   z = x W^T + bias        y = act(z) + residual
//   dz = dy act'(z)         dx = dz W      dW = dz^T x      dbias = sum over the batch of dz
//
// x [B][IC], W [OC][IC], z, y, dy [B][OC]; products are summed in 32 bits. dz is rounded once
// to the operands' type, because it is an operand of the two products that follow; dbias sums
// it before that rounding.
#include <cmath>

#include "ito_float.cuh"

namespace ito {

// ----------------------------------------------------------------- activations

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

// What the product's epilogue does with a sum.
struct FpEpilogue {
    const void* bias;
    int bias_type, act;
    const void* residual;
    int64_t ldr;
    int out_type;          // of y and residual
    void* y;
    int64_t ldy;
    void* z;               // the operands' type, may be null
    int64_t ldz;
};

template <typename T>
__device__ __forceinline__ void fp_finish(const FpEpilogue& e, int64_t r, int64_t c, float v)
{
    if (e.bias) v += load_typed(e.bias, e.bias_type, c);
    if (e.z) static_cast<T*>(e.z)[r * e.ldz + c] = from_f32<T>(v);
    v = act_value(e.act, v);
    if (e.residual) v += load_typed(e.residual, e.out_type, r * e.ldr + c);
    if (e.out_type == ITO_F32) static_cast<float*>(e.y)[r * e.ldy + c] = v;
    else static_cast<T*>(e.y)[r * e.ldy + c] = from_f32<T>(v);
}

// ------------------------------------------------------------ the product, simply

// C[m][n] = sum_k A(m, k) B(n, k), A(m, k) = A[m sam + k sak], B(n, k) = B[n sbn + k sbk]:
// 64 x 64 tiles, 16 of K at a time in shared memory, 4 x 4 sums to a thread.
template <typename T>
__global__ void __launch_bounds__(256)
    k_fp_product(const T* __restrict__ A, int64_t sam, int64_t sak, const T* __restrict__ B, int64_t sbn, int64_t sbk,
                 int M, int N, int K, const FpEpilogue e)
{
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float sa[16][65], sb[16][65];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int tiles_n = (N + 63) / 64;
    const int64_t tiles = (int64_t)((M + 63) / 64) * tiles_n;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int m0 = (int)(t / tiles_n) * 64, n0 = (int)(t % tiles_n) * 64;
        float acc[4][4] = {};
        for (int k0 = 0; k0 < K; k0 += 16) {
            for (int i = threadIdx.x; i < 1024; i += 256) {
                const int r = sak == 1 ? i >> 4 : i & 63, c = sak == 1 ? i & 15 : i >> 6;
                sa[c][r] = m0 + r < M && k0 + c < K ? to_f32(A[(m0 + r) * sam + (k0 + c) * sak]) : 0.0f;
                const int r2 = sbk == 1 ? i >> 4 : i & 63, c2 = sbk == 1 ? i & 15 : i >> 6;
                sb[c2][r2] = n0 + r2 < N && k0 + c2 < K ? to_f32(B[(n0 + r2) * sbn + (k0 + c2) * sbk]) : 0.0f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 16; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty + 16 * i] * sb[k][tx + 16 * j];
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j)
                if (m0 + ty + 16 * i < M && n0 + tx + 16 * j < N)
                    fp_finish<T>(e, m0 + ty + 16 * i, n0 + tx + 16 * j, acc[i][j]);
    }
}

// dz = dy act'(z), rounded to T, and the columns' sums of the unrounded dz over rows
// [blockIdx.y rows_per, ...), each share in its own row of the partials.
template <typename T>
__global__ void __launch_bounds__(256)
    k_fp_dz(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ z, int64_t ldz, int act, int B, int OC,
            int rows_per, T* __restrict__ dz, int64_t lddz, float* __restrict__ part)
{
    griddep_wait();
    griddep_launch_dependents();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= OC) return;
    const int r1 = min(B, ((int)blockIdx.y + 1) * rows_per);
    float s = 0.0f;
    for (int r = blockIdx.y * rows_per; r < r1; ++r) {
        float v = to_f32(dy[r * lddy + c]);
        if (act != ITO_ACT_NONE) v *= act_slope(act, to_f32(z[r * ldz + c]));
        s += v;
        if (dz) dz[r * lddz + c] = from_f32<T>(v);
    }
    if (part) part[(int64_t)blockIdx.y * OC + c] = s;
}

__global__ void __launch_bounds__(256)
    k_fp_column_sums(const float* __restrict__ part, int parts, int n, float* __restrict__ out)
{
    griddep_wait();
    griddep_launch_dependents();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= n) return;
    float s = 0.0f;
    for (int p = 0; p < parts; ++p) s += part[(int64_t)p * n + c];
    out[c] = s;
}

constexpr int kDzParts = 64;         // shares of the batch in the bias gradient's sum

static int dz_rows_per(int B) { return (B + kDzParts - 1) / kDzParts; }
static int dz_parts(int B) { return (B + dz_rows_per(B) - 1) / dz_rows_per(B); }
static size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

static int check_sizes(int B, int IC, int OC)
{
    if (B < 1 || IC < 1 || OC < 1) return set_error(ITO_ERR_SHAPE, "sizes must be >= 1");
    if (B > (1 << 20) || IC > (1 << 20) || OC > (1 << 20)) return set_error(ITO_ERR_SHAPE, "a size above 2^20");
    return ITO_OK;
}

static int check_tensor(const void* p, int type, int64_t ld, int rows, int cols, const char* name)
{
    if (!aligned_to(p, type_bytes(type))) return set_error(ITO_ERR_ARG, "%s: misaligned pointer", name);
    if (rows > 1 && ld < cols) return set_error(ITO_ERR_SHAPE, "%s: row stride below its columns", name);
    return ITO_OK;
}

static int check_types(int type, int out_type, int act)
{
    if (type != ITO_BF16 && type != ITO_F16) return set_error(ITO_ERR_ARG, "type must be ITO_BF16 or ITO_F16");
    if (out_type != type && out_type != ITO_F32) return set_error(ITO_ERR_ARG, "out_type must be type or ITO_F32");
    if (act < ITO_ACT_NONE || act > ITO_ACT_SILU) return set_error(ITO_ERR_ARG, "unknown activation");
    return ITO_OK;
}

static int check_ws(const void* ws, size_t bytes, size_t need)
{
    if (!need) return ITO_OK;
    if (!ws) return set_error(ITO_ERR_ARG, "workspace is NULL");
    if (!aligned_to(ws, 256)) return set_error(ITO_ERR_ARG, "workspace not 256-byte aligned");
    if (bytes < need) return set_error(ITO_ERR_ARG, "workspace too small");
    return ITO_OK;
}

template <typename T>
static int product(const void* A, int64_t sam, int64_t sak, const void* B, int64_t sbn, int64_t sbk, int M, int N,
                   int K, const FpEpilogue& e, cudaStream_t s)
{
    const int64_t tiles = (int64_t)((M + 63) / 64) * ((N + 63) / 64);
    launch_pdl(k_fp_product<T>, (unsigned)(tiles < 65535 ? tiles : 65535), 256, 0, s, static_cast<const T*>(A), sam,
               sak, static_cast<const T*>(B), sbn, sbk, M, N, K, e);
    return launch_status("linear");
}

template <typename T>
static int run_bwd(const void* dy, int64_t lddy, const void* z, int64_t ldz, const void* x, int64_t ldx,
                   const void* W, int64_t ldw, int type, int out_type, int act, int B, int IC, int OC, void* ws,
                   void* dx, int64_t lddx, void* dW, int64_t lddw, float* dbias, cudaStream_t s)
{
    T* dz = static_cast<T*>(ws);
    const int64_t lddz = pad8(OC);
    float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + align256((size_t)B * lddz * 2));
    launch_pdl(k_fp_dz<T>, dim3((OC + 255) / 256, dz_parts(B)), 256, 0, s, static_cast<const T*>(dy), lddy,
               static_cast<const T*>(z), ldz, act, B, OC, dz_rows_per(B), dz, lddz, part);
    if (dbias) launch_pdl(k_fp_column_sums, (OC + 255) / 256, 256, 0, s, part, dz_parts(B), OC, dbias);
    int r = launch_status("linear backward");
    if (!r && dx)
        r = product<T>(dz, lddz, 1, W, 1, ldw, B, IC, OC,
                       FpEpilogue{nullptr, 0, 0, nullptr, 0, type, dx, lddx, nullptr, 0}, s);
    if (!r && dW)
        r = product<T>(dz, 1, lddz, x, 1, ldx, OC, IC, B, FpEpilogue{nullptr, 0, 0, nullptr, 0, out_type, dW, lddw, nullptr, 0}, s);
    return r;
}

}  // namespace ito

using namespace ito;

extern "C" {

size_t ito_fp_linear_fwd_workspace_size(const void* x, int64_t ldx, const void* W, int64_t ldw, int B, int IC, int OC)
{
    (void)x; (void)ldx; (void)W; (void)ldw;
    if (check_sizes(B, IC, OC)) return 0;
    return 0;
}

int ito_fp_linear_fwd(const void* x, int64_t ldx, const void* W, int64_t ldw, const void* bias, const void* residual,
                      int64_t ldr, int type, int out_type, int bias_type, int act, int B, int IC, int OC,
                      void* workspace, size_t workspace_bytes, void* z, int64_t ldz, void* y, int64_t ldy,
                      void* stream)
{
    if (!x || !W || !y) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    int r = check_types(type, out_type, act);
    if (!r) r = check_sizes(B, IC, OC);
    if (r) return r;
    if (bias && bias_type != type && bias_type != ITO_F32)
        return set_error(ITO_ERR_ARG, "bias_type must be type or ITO_F32");
    r = check_tensor(x, type, ldx, B, IC, "x");
    if (!r) r = check_tensor(W, type, ldw, OC, IC, "W");
    if (!r && bias) r = check_tensor(bias, bias_type, OC, 1, OC, "bias");
    if (!r && residual) r = check_tensor(residual, out_type, ldr, B, OC, "residual");
    if (!r && z) r = check_tensor(z, type, ldz, B, OC, "z");
    if (!r) r = check_tensor(y, out_type, ldy, B, OC, "y");
    if (!r) r = check_ws(workspace, workspace_bytes, ito_fp_linear_fwd_workspace_size(x, ldx, W, ldw, B, IC, OC));
    if (r) return r;
    const FpEpilogue e{bias, bias_type, act, residual, ldr, out_type, y, ldy, z, ldz};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (type == ITO_BF16) return product<__nv_bfloat16>(x, ldx, 1, W, ldw, 1, B, OC, IC, e, s);
    return product<__half>(x, ldx, 1, W, ldw, 1, B, OC, IC, e, s);
}

size_t ito_fp_linear_bwd_workspace_size(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* W,
                                        int64_t ldw, int act, int B, int IC, int OC)
{
    (void)dy; (void)lddy; (void)x; (void)ldx; (void)W; (void)ldw; (void)act;
    if (check_sizes(B, IC, OC)) return 0;
    return align256((size_t)B * pad8(OC) * 2) + align256((size_t)dz_parts(B) * OC * 4);
}

int ito_fp_linear_bwd(const void* dy, int64_t lddy, const void* z, int64_t ldz, const void* x, int64_t ldx,
                      const void* W, int64_t ldw, int type, int out_type, int act, int B, int IC, int OC,
                      void* workspace, size_t workspace_bytes, void* dx, int64_t lddx, void* dW, int64_t lddw,
                      float* dbias, void* stream)
{
    if (!dy || (dW && !x) || (dx && !W)) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    if (!dx && !dW && !dbias) return set_error(ITO_ERR_ARG, "no output");
    int r = check_types(type, out_type, act);
    if (!r) r = check_sizes(B, IC, OC);
    if (r) return r;
    if (act != ITO_ACT_NONE && !z) return set_error(ITO_ERR_ARG, "an activation's gradient needs z");
    r = check_tensor(dy, type, lddy, B, OC, "dy");
    if (!r && act != ITO_ACT_NONE) r = check_tensor(z, type, ldz, B, OC, "z");
    if (!r && dW) r = check_tensor(x, type, ldx, B, IC, "x");
    if (!r && dx) r = check_tensor(W, type, ldw, OC, IC, "W");
    if (!r && dx) r = check_tensor(dx, type, lddx, B, IC, "dx");
    if (!r && dW) r = check_tensor(dW, out_type, lddw, OC, IC, "dW");
    if (!r && !aligned_to(dbias, 4)) r = set_error(ITO_ERR_ARG, "dbias: misaligned pointer");
    if (!r)
        r = check_ws(workspace, workspace_bytes,
                     ito_fp_linear_bwd_workspace_size(dy, lddy, x, ldx, W, ldw, act, B, IC, OC));
    if (r) return r;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (type == ITO_BF16)
        return run_bwd<__nv_bfloat16>(dy, lddy, z, ldz, x, ldx, W, ldw, type, out_type, act, B, IC, OC, workspace, dx,
                                      lddx, dW, lddw, dbias, s);
    return run_bwd<__half>(dy, lddy, z, ldz, x, ldx, W, ldw, type, out_type, act, B, IC, OC, workspace, dx, lddx, dW,
                           lddw, dbias, s);
}

}  // extern "C"
