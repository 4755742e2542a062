// Layer norm over the last dimension, forward and backward.
//
//   mean = sum x / n      rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)      h = (x - mean) rstd
//   y = h gamma + beta
//   a = dy gamma;  dx = rstd (a - sum(a) / n - h sum(a h) / n)
//   dgamma = sum over rows of dy h;  dbeta = sum over rows of dy
//
// The variance is taken from the centred values (a second pass over the row), not as the
// difference of two large sums. Sums are held in 32 bits.
#include "ito_float.cuh"

namespace ito {

constexpr int kLnThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kLnThreads)
    k_layer_norm_fwd(const T* __restrict__ x, int64_t ldx, const void* __restrict__ gamma,
                     const void* __restrict__ beta, int w_type, int64_t rows, int cols, float eps, T* __restrict__ y,
                     int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd)
{
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* xr = x + r * ldx;
        float s = 0.0f;
        for (int c = threadIdx.x; c < cols; c += kLnThreads) s += to_f32(xr[c]);
        const float mu = block_reduce(s, AddOp()) / (float)cols;
        float q = 0.0f;
        for (int c = threadIdx.x; c < cols; c += kLnThreads) {
            const float d = to_f32(xr[c]) - mu;
            q += d * d;
        }
        const float rs = 1.0f / sqrtf(block_reduce(q, AddOp()) / (float)cols + eps);
        for (int c = threadIdx.x; c < cols; c += kLnThreads) {
            const float h = (to_f32(xr[c]) - mu) * rs;
            const float g = gamma ? load_typed(gamma, w_type, c) : 1.0f;
            const float b = beta ? load_typed(beta, w_type, c) : 0.0f;
            y[r * ldy + c] = from_f32<T>(h * g + b);
        }
        if (threadIdx.x == 0) {
            if (mean) mean[r] = mu;
            if (rstd) rstd[r] = rs;
        }
    }
}

// dx, and this CTA's share of dgamma and dbeta: rows blockIdx.x, + gridDim.x, ... summed
// into its own row of the partials, which k_layer_norm_wgrad adds in a fixed order.
template <typename T>
__global__ void __launch_bounds__(kLnThreads)
    k_layer_norm_bwd(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x, int64_t ldx,
                     const void* __restrict__ gamma, int w_type, const float* __restrict__ mean,
                     const float* __restrict__ rstd, int64_t rows, int cols, T* __restrict__ dx, int64_t lddx,
                     float* __restrict__ part)
{
    griddep_wait();
    griddep_launch_dependents();
    float* pg = part ? part + (int64_t)blockIdx.x * 2 * cols : nullptr;
    float* pb = part ? pg + cols : nullptr;
    bool first = true;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const float mu = mean[r], rs = rstd[r];
        float sa = 0.0f, sh = 0.0f;
        for (int c = threadIdx.x; c < cols; c += kLnThreads) {
            const float d = to_f32(dy[r * lddy + c]);
            const float h = (to_f32(x[r * ldx + c]) - mu) * rs;
            const float a = d * (gamma ? load_typed(gamma, w_type, c) : 1.0f);
            sa += a;
            sh += a * h;
            if (part) {
                pg[c] = (first ? 0.0f : pg[c]) + d * h;
                pb[c] = (first ? 0.0f : pb[c]) + d;
            }
        }
        first = false;
        if (!dx) continue;
        sa = block_reduce(sa, AddOp()) / (float)cols;
        sh = block_reduce(sh, AddOp()) / (float)cols;
        for (int c = threadIdx.x; c < cols; c += kLnThreads) {
            const float h = (to_f32(x[r * ldx + c]) - mu) * rs;
            const float a = to_f32(dy[r * lddy + c]) * (gamma ? load_typed(gamma, w_type, c) : 1.0f);
            dx[r * lddx + c] = from_f32<T>(rs * (a - sa - h * sh));
        }
    }
}

__global__ void __launch_bounds__(kLnThreads)
    k_layer_norm_wgrad(const float* __restrict__ part, int parts, int cols, float* __restrict__ dgamma,
                       float* __restrict__ dbeta)
{
    griddep_wait();
    griddep_launch_dependents();
    for (int c = blockIdx.x * kLnThreads + threadIdx.x; c < cols; c += gridDim.x * kLnThreads) {
        float g = 0.0f, b = 0.0f;
        for (int p = 0; p < parts; ++p) {
            g += part[(int64_t)p * 2 * cols + c];
            b += part[(int64_t)p * 2 * cols + cols + c];
        }
        if (dgamma) dgamma[c] = g;
        if (dbeta) dbeta[c] = b;
    }
}

static int ln_parts(int64_t rows) { return rows < 2 * kNumSMsHint ? (int)rows : 2 * kNumSMsHint; }

static int check_ln(const void* x, int64_t ldx, int type, int64_t rows, int cols, const char* name)
{
    if (!aligned_to(x, type_bytes(type))) return set_error(ITO_ERR_ARG, "%s: misaligned pointer", name);
    if (rows > 1 && ldx < cols) return set_error(ITO_ERR_SHAPE, "%s: row stride below cols", name);
    return ITO_OK;
}

static int check_ln_sizes(int type, int w_type, bool weighted, int64_t rows, int cols)
{
    if (!type_known(type)) return set_error(ITO_ERR_ARG, "unknown type");
    if (weighted && w_type != ITO_F32 && w_type != type)
        return set_error(ITO_ERR_ARG, "w_type must be ITO_F32 or the tensors' type");
    if (rows < 1 || cols < 1) return set_error(ITO_ERR_SHAPE, "sizes must be >= 1");
    if (rows > (int64_t(1) << 40) || cols > (1 << 24)) return set_error(ITO_ERR_SHAPE, "rows above 2^40 or cols above 2^24");
    return ITO_OK;
}

template <typename T>
static int run_fwd(const void* x, int64_t ldx, const void* gamma, const void* beta, int w_type, int64_t rows,
                   int cols, float eps, void* y, int64_t ldy, float* mean, float* rstd, cudaStream_t s)
{
    const int64_t grid = rows < 8 * num_sms() ? rows : 8 * num_sms();
    launch_pdl(k_layer_norm_fwd<T>, (unsigned)grid, kLnThreads, 0, s, static_cast<const T*>(x), ldx, gamma, beta,
               w_type, rows, cols, eps, static_cast<T*>(y), ldy, mean, rstd);
    return launch_status("layer norm");
}

template <typename T>
static int run_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* gamma, int w_type,
                   const float* mean, const float* rstd, int64_t rows, int cols, float* part, void* dx, int64_t lddx,
                   float* dgamma, float* dbeta, cudaStream_t s)
{
    const int parts = ln_parts(rows);
    launch_pdl(k_layer_norm_bwd<T>, parts, kLnThreads, 0, s, static_cast<const T*>(dy), lddy,
               static_cast<const T*>(x), ldx, gamma, w_type, mean, rstd, rows, cols, static_cast<T*>(dx), lddx,
               dgamma || dbeta ? part : static_cast<float*>(nullptr));
    if (dgamma || dbeta)
        launch_pdl(k_layer_norm_wgrad, (cols + kLnThreads - 1) / kLnThreads, kLnThreads, 0, s, part, parts, cols,
                   dgamma, dbeta);
    return launch_status("layer norm");
}

}  // namespace ito

using namespace ito;

extern "C" {

int ito_layer_norm_fwd(const void* x, int64_t ldx, int type, const void* gamma, const void* beta, int w_type,
                       int64_t rows, int cols, float eps, void* y, int64_t ldy, float* mean, float* rstd,
                       void* stream)
{
    if (!x || !y) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    int r = check_ln_sizes(type, w_type, gamma || beta, rows, cols);
    if (!r) r = check_ln(x, ldx, type, rows, cols, "x");
    if (!r) r = check_ln(y, ldy, type, rows, cols, "y");
    if (r) return r;
    if (!(eps >= 0.0f)) return set_error(ITO_ERR_ARG, "eps must be >= 0");
    if (!aligned_to(gamma, type_bytes(w_type)) || !aligned_to(beta, type_bytes(w_type)) || !aligned_to(mean, 4) ||
        !aligned_to(rstd, 4))
        return set_error(ITO_ERR_ARG, "misaligned pointer");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (type == ITO_F32) return run_fwd<float>(x, ldx, gamma, beta, w_type, rows, cols, eps, y, ldy, mean, rstd, s);
    if (type == ITO_BF16)
        return run_fwd<__nv_bfloat16>(x, ldx, gamma, beta, w_type, rows, cols, eps, y, ldy, mean, rstd, s);
    return run_fwd<__half>(x, ldx, gamma, beta, w_type, rows, cols, eps, y, ldy, mean, rstd, s);
}

size_t ito_layer_norm_bwd_workspace_size(int64_t rows, int cols)
{
    if (rows < 1 || cols < 1 || rows > (int64_t(1) << 40) || cols > (1 << 24)) return 0;
    return (size_t)ln_parts(rows) * 2 * cols * sizeof(float);
}

int ito_layer_norm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, int type, const void* gamma,
                       int w_type, const float* mean, const float* rstd, int64_t rows, int cols, void* workspace,
                       size_t workspace_bytes, void* dx, int64_t lddx, float* dgamma, float* dbeta, void* stream)
{
    if (!dy || !x || !mean || !rstd) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    if (!dx && !dgamma && !dbeta) return set_error(ITO_ERR_ARG, "no output");
    int r = check_ln_sizes(type, w_type, gamma, rows, cols);
    if (!r) r = check_ln(dy, lddy, type, rows, cols, "dy");
    if (!r) r = check_ln(x, ldx, type, rows, cols, "x");
    if (!r && dx) r = check_ln(dx, lddx, type, rows, cols, "dx");
    if (r) return r;
    if (!aligned_to(gamma, type_bytes(w_type)) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) ||
        !aligned_to(dgamma, 4) || !aligned_to(dbeta, 4))
        return set_error(ITO_ERR_ARG, "misaligned pointer");
    if (dgamma || dbeta) {
        if (!workspace) return set_error(ITO_ERR_ARG, "workspace is NULL");
        if (!aligned_to(workspace, 256)) return set_error(ITO_ERR_ARG, "workspace not 256-byte aligned");
        if (workspace_bytes < ito_layer_norm_bwd_workspace_size(rows, cols))
            return set_error(ITO_ERR_ARG, "workspace too small");
    }
    float* part = static_cast<float*>(workspace);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (type == ITO_F32)
        return run_bwd<float>(dy, lddy, x, ldx, gamma, w_type, mean, rstd, rows, cols, part, dx, lddx, dgamma, dbeta, s);
    if (type == ITO_BF16)
        return run_bwd<__nv_bfloat16>(dy, lddy, x, ldx, gamma, w_type, mean, rstd, rows, cols, part, dx, lddx, dgamma,
                                      dbeta, s);
    return run_bwd<__half>(dy, lddy, x, ldx, gamma, w_type, mean, rstd, rows, cols, part, dx, lddx, dgamma, dbeta, s);
}

}  // extern "C"
