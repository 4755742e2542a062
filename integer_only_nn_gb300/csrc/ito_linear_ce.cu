// Cross entropy of a linear layer's classes (a head over a large vocabulary) and its gradient,
// without the logits in memory.
//
//   l_j = x W_j        lse = log sum_j exp(l_j)        loss = lse - l_target
//   dl_j = g_loss (p_j - hot_j) + g_lse p_j,   p = exp(l - lse)        dx = dl W        dW = dl^T x
//
// Forward the product's epilogue keeps, for each row and the columns of a tile that a warp drains,
// the largest sum and the sum of exponentials (8 bytes for 64 to 128 logits), and the target's
// logit; a second kernel joins them. Logits are never rounded to 16 bits.
//
// Backward goes through the vocabulary in pieces: a piece's logits are computed again, by the kernel that the
// forward pass had and in the same order, so that they are what went into lse in every bit (p - 1 of a target with nearly
// all of the probability is a difference of neighbours). Their epilogue leaves dl in the operands' type (rounded
// once; it is an operand of the two products that follow), then dx's and dW's products of the piece share a launch.
// dx is added up over the pieces in 32 bits and rounded at the last one. Of a few rows the products stream W
// (ito_fp_few_grad.cu).
#include "ito_fp_rows.cuh"

namespace ito {

// -------------------------------------------------------------- forward's join

// A block joins the parts of R rows (a power of two): thread t those of row t % R, every
// (threads / R)-th; then halves of the block meet, always in the same order.
constexpr int kCeJoinThreads = 512;

__global__ void __launch_bounds__(kCeJoinThreads)
    k_ce_join(const float2* __restrict__ part, int parts, int rows, int R, const float* __restrict__ hit,
              const int32_t* __restrict__ targets, int classes, float* __restrict__ loss, float* __restrict__ lse, int* err)
{
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float ms[kCeJoinThreads], ss[kCeJoinThreads];
    const int t = threadIdx.x, slots = kCeJoinThreads / R, row = blockIdx.x * R + t % R;
    float m = -INFINITY, s = 0.0f;
    if (row < rows) {
        constexpr int U = 4;                 // parts whose loads are in flight together
        for (int p = t / R; p < parts; p += slots * U) {
            float2 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = p + u * slots;
                v[u] = q < parts ? part[(int64_t)q * rows + row] : make_float2(-INFINITY, 0.0f);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) fp_softmax_add(m, s, v[u].x, v[u].y);
        }
    }
    ms[t] = m;
    ss[t] = s;
    for (int o = kCeJoinThreads / 2; o >= R; o >>= 1) {
        __syncthreads();
        if (t < o) {
            fp_softmax_add(m, s, ms[t + o], ss[t + o]);
            ms[t] = m;
            ss[t] = s;
        }
    }
    if (t >= R || row >= rows) return;
    // (s is 0 where every logit is -inf, and lse -inf)
    const float l = m + logf(s);
    if (lse) lse[row] = l;
    const int target = targets[row];
    const bool in = target >= 0 && target < classes;
    if (!in && target != -1) raise_device_error(err, ITO_ERR_ARG);
    if (loss) loss[row] = !in ? 0.0f : s == 0.0f ? INFINITY : l - hit[row];
}

// ---------------------------------------------------------- backward's scale

// float16 has no room below 6e-8 for the gradients of rare classes: dl carries a power of two that
// brings the largest |g| to 2^12 .. 2^13, and the products' sums are multiplied by its inverse. What rows without
// a token hold in g_loss does not count. (The factor and its inverse are both normal floats: 2^-115 for the largest |g|,
// 2^126 at most, which leaves those below 2^-114 less than that.)
// out: [2] that factor and its inverse
__global__ void __launch_bounds__(1024)
    k_ce_scale(const float* __restrict__ g_loss, const float* __restrict__ g_lse, const int32_t* __restrict__ targets,
               int classes, int rows, float* __restrict__ out)
{
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float most[32];
    float m = 0.0f;
#pragma unroll 4
    for (int r = threadIdx.x; r < rows; r += blockDim.x) {
        const int t = targets[r];
        const float g = fabsf(g_loss[r]);
        m = fmaxf(m, (t >= 0 && t < classes ? g : 0.0f) + (g_lse ? fabsf(g_lse[r]) : 0.0f));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x) return;
    for (int w = 1; w < 32; ++w) m = fmaxf(m, most[w]);
    int e = 0;
    if (m > 0.0f && m < INFINITY) {
        frexpf(m, &e);                       // m = f 2^e, f in [1/2, 1)
        e = min(13 - e, 126);               // (e is 128 at most)
    }
    out[0] = ldexpf(1.0f, e);
    out[1] = ldexpf(1.0f, -e);
}

// ------------------------------------------------------------------------ host

// Classes of a piece: dl of a piece takes 256 MB at most, in whole tiles of 256 columns.
constexpr int64_t kCePieceBytes = 256 << 20;

static int ce_piece(int rows, int classes)
{
    const int64_t n = kCePieceBytes / 2 / rows / 256 * 256;
    return (int)std::min<int64_t>(classes, std::max<int64_t>(n, 256));
}

// a row of dl: whole lines of 128 bytes, which is what the products' loads take of it at a time
static int64_t ce_ldl(int64_t piece) { return (piece + 63) & ~int64_t(63); }

static int ce_parts(int rows, int d, int classes, bool few)
{
    if (few) return (classes + 15) / 16;
    return std::max(1, fp_loss_parts(rows, classes, d));
}

// Backward of a few rows, which are in one piece (32 rows: up to 2^22 classes): the products stream W (fp_few_grad), and
// the logits where the forward pass's did. Where both do, W and x are read as they are (5 x 787 x 50001 f16, us: 101;
// with copies and all in tiles 142).
struct CeFew {
    bool grad, logits;
};
static CeFew ce_few(const void* x, int64_t ldx, const void* W, int64_t ldw, int rows, int d, int classes)
{
    return CeFew{fp_few_grad_rows(rows), fp_few_logits(rows, d, classes, fp_rows_vec(x, ldx, W, ldw, rows, d, classes))};
}

// of a piece of n classes
static size_t ce_products_bytes(int rows, int d, int classes, int n)
{
    return std::max(fp_gemm_ws_bytes(rows, n, d, false, FpEnd::DLogits, 1, classes),
                    fp_gemm_ws_bytes(rows, d, n, true, FpEnd::Grad) + fp_gemm_ws_bytes(n, d, rows, true, FpEnd::Grad));
}

static int check_ce(int type, const void* x, int64_t ldx, const void* W, int64_t ldw, const int32_t* targets, int rows,
                    int d, int classes)
{
    if (!x || !W || !targets) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    int r = fp_check_types(type, type, ITO_ACT_NONE);
    if (!r) r = fp_check_sizes(rows, d, classes);
    if (!r) r = fp_check_tensor(x, type, ldx, rows, d, "x");
    if (!r) r = fp_check_tensor(W, type, ldw, classes, d, "W");
    if (!r && !aligned_to(targets, 4)) r = set_error(ITO_ERR_ARG, "targets: misaligned pointer");
    return r;
}

}  // namespace ito

using namespace ito;

extern "C" {

size_t ito_linear_cross_entropy_fwd_workspace_size(const void* x, int64_t ldx, const void* W, int64_t ldw, int rows,
                                                   int d, int classes)
{
    if (fp_check_sizes(rows, d, classes)) return 0;
    const bool few = fp_few_logits(rows, d, classes, fp_rows_vec(x, ldx, W, ldw, rows, d, classes));
    const size_t own = align256((size_t)ce_parts(rows, d, classes, few) * rows * 8) + align256((size_t)rows * 4);
    if (few) return own;
    return own + fp_copy_bytes(x, ldx, rows, d) + fp_copy_bytes(W, ldw, classes, d) +
           fp_gemm_ws_bytes(rows, classes, d, false, FpEnd::Loss);
}

int ito_linear_cross_entropy_fwd(const void* x, int64_t ldx, const void* W, int64_t ldw, int type,
                                 const int32_t* targets, int rows, int d, int classes, void* workspace,
                                 size_t workspace_bytes, float* loss, float* lse, void* stream)
{
    int r = check_ce(type, x, ldx, W, ldw, targets, rows, d, classes);
    if (!r && !loss && !lse) r = set_error(ITO_ERR_ARG, "no output");
    if (!r && (!aligned_to(loss, 4) || !aligned_to(lse, 4))) r = set_error(ITO_ERR_ARG, "misaligned result pointer");
    if (!r)
        r = fp_check_ws(workspace, workspace_bytes,
                        ito_linear_cross_entropy_fwd_workspace_size(x, ldx, W, ldw, rows, d, classes));
    if (r) return r;
    int* err = device_error_word();
    if (!err) return set_error(ITO_ERR_CUDA, "device error word unavailable");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool few = fp_few_logits(rows, d, classes, fp_rows_vec(x, ldx, W, ldw, rows, d, classes));
    const int parts = ce_parts(rows, d, classes, few);
    char* ws = static_cast<char*>(workspace);
    FpMore more{};
    more.targets = targets;
    more.classes = classes;
    more.part = reinterpret_cast<float2*>(ws);
    ws += align256((size_t)parts * rows * 8);
    more.hit = reinterpret_cast<float*>(ws);
    ws += align256((size_t)rows * 4);
    FpEpilogue e{};
    e.type = e.out_type = type;
    if (few) {
        r = fp_run_rows<FpEnd::Loss>(x, ldx, W, ldw, nullptr, 0, rows, d, classes, e, more, s);
    } else {
        FpCopy copies{};
        const void* xa = fp_aligned_operand(x, &ldx, rows, d, &ws, &copies);
        const void* wa = fp_aligned_operand(W, &ldw, classes, d, &ws, &copies);
        r = fp_run_copies(copies, s);
        if (r) return r;
        const FpProduct p{FpOperand{xa, ldx, false}, FpOperand{wa, ldw, false}, rows, classes, d, e, FpEnd::Loss, more};
        r = fp_gemm(&p, 1, ws, s);
    }
    if (r) return r;
    int R = 1;
    while (R < 32 && R * num_sms() < rows) R *= 2;
    launch_pdl(k_ce_join, (rows + R - 1) / R, kCeJoinThreads, 0, s, more.part, parts, rows, R, more.hit, targets, classes,
               loss, lse, err);
    return launch_status("linear cross entropy");
}

size_t ito_linear_cross_entropy_bwd_workspace_size(const void* x, int64_t ldx, const void* W, int64_t ldw, int rows,
                                                   int d, int classes)
{
    if (fp_check_sizes(rows, d, classes)) return 0;
    const int piece = ce_piece(rows, classes), last = (classes - 1) % piece + 1;
    const CeFew few = ce_few(x, ldx, W, ldw, rows, d, classes);
    size_t n = 256 + align256((size_t)rows * ce_ldl(piece) * 2);
    if (!few.logits || !few.grad) n += fp_copy_bytes(x, ldx, rows, d) + fp_copy_bytes(W, ldw, classes, d);
    if (few.grad)
        return n + std::max(few.logits ? 0 : fp_gemm_ws_bytes(rows, classes, d, false, FpEnd::DLogits),
                            fp_few_grad_ws_bytes(rows, classes, d, 1));
    if (piece < classes) n += align256((size_t)rows * pad4(d) * 4);
    return n + std::max(ce_products_bytes(rows, d, classes, piece), ce_products_bytes(rows, d, classes, last));
}

int ito_linear_cross_entropy_bwd(const void* x, int64_t ldx, const void* W, int64_t ldw, int type,
                                 const int32_t* targets, const float* lse, const float* g_loss, const float* g_lse,
                                 int out_type, int rows, int d, int classes, void* workspace, size_t workspace_bytes,
                                 void* dx, int64_t lddx, void* dW, int64_t lddw, void* stream)
{
    if (!lse || !g_loss) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    if (!dx && !dW) return set_error(ITO_ERR_ARG, "no output");
    int r = check_ce(type, x, ldx, W, ldw, targets, rows, d, classes);
    if (!r) r = fp_check_types(type, out_type, ITO_ACT_NONE);
    if (!r && (!aligned_to(lse, 4) || !aligned_to(g_loss, 4) || !aligned_to(g_lse, 4)))
        r = set_error(ITO_ERR_ARG, "misaligned pointer");
    if (!r && dx) r = fp_check_tensor(dx, type, lddx, rows, d, "dx");
    if (!r && dW) r = fp_check_tensor(dW, out_type, lddw, classes, d, "dW");
    if (!r)
        r = fp_check_ws(workspace, workspace_bytes,
                        ito_linear_cross_entropy_bwd_workspace_size(x, ldx, W, ldw, rows, d, classes));
    if (r) return r;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int piece = ce_piece(rows, classes);
    char* ws = static_cast<char*>(workspace);
    float* scale = nullptr;
    if (type == ITO_F16) {
        scale = reinterpret_cast<float*>(ws);
        launch_pdl(k_ce_scale, 1, 1024, 0, s, g_loss, g_lse, targets, classes, rows, scale);
        r = launch_status("linear cross entropy backward");
        if (r) return r;
    }
    ws += 256;
    const CeFew few = ce_few(x, ldx, W, ldw, rows, d, classes);
    const void* xa = x;
    const uint16_t* wa = static_cast<const uint16_t*>(W);
    if (!few.logits || !few.grad) {
        FpCopy copies{};
        xa = fp_aligned_operand(x, &ldx, rows, d, &ws, &copies);
        wa = static_cast<const uint16_t*>(fp_aligned_operand(W, &ldw, classes, d, &ws, &copies));
        r = fp_run_copies(copies, s);
        if (r) return r;
    }
    void* dl = ws;
    const int64_t ldl = ce_ldl(piece);
    ws += align256((size_t)rows * ldl * 2);
    float* acc = nullptr;
    if (piece < classes) {
        acc = reinterpret_cast<float*>(ws);
        ws += align256((size_t)rows * pad4(d) * 4);
    }
    const size_t out_bytes = type_bytes(out_type);
    for (int first = 0; first < classes; first += piece) {
        const int n = std::min(piece, classes - first);
        const bool last = first + n == classes;
        const uint16_t* w = wa + (int64_t)first * ldw;
        FpEpilogue e{};
        e.type = e.out_type = type;
        e.y = dl;
        e.ldy = ldl;
        FpProduct logits{FpOperand{xa, ldx, false}, FpOperand{w, ldw, false}, rows, n, d, e, FpEnd::DLogits};
        logits.x.targets = targets;
        logits.x.first = first;
        logits.x.classes = classes;
        logits.x.lse = lse;
        logits.x.g_loss = g_loss;
        logits.x.g_lse = g_lse;
        logits.x.scale = scale;
        logits.plan_n = classes;
        r = few.logits ? fp_run_rows<FpEnd::DLogits>(xa, ldx, w, ldw, nullptr, 0, rows, d, n, e, logits.x, s)
                       : fp_gemm(&logits, 1, ws, s);
        if (r) return r;
        if (few.grad) {
            const FpFewGrad p{{static_cast<const uint16_t*>(dl)}, ldl, {w}, {ldw}, static_cast<const uint16_t*>(xa), ldx,
                              type, out_type, rows, n, d, scale ? scale + 1 : nullptr, dx, lddx, {dW}, {lddw}};
            return fp_few_grad(p, ws, s);
        }
        FpProduct products[2];
        int k = 0;
        if (dx) {
            FpEpilogue o{};
            o.type = type;
            o.out_type = last ? type : ITO_F32;
            o.y = last ? dx : acc;
            o.ldy = last ? lddx : pad4(d);
            FpProduct p{FpOperand{dl, ldl, false}, FpOperand{w, ldw, true}, rows, d, n, o, FpEnd::Grad};
            p.x.alpha = scale ? scale + 1 : nullptr;
            p.x.acc = first ? acc : nullptr;
            p.x.ldacc = pad4(d);
            products[k++] = p;
        }
        if (dW) {
            FpEpilogue o{};
            o.type = type;
            o.out_type = out_type;
            o.y = static_cast<char*>(dW) + (int64_t)first * lddw * out_bytes;
            o.ldy = lddw;
            FpProduct p{FpOperand{dl, ldl, true}, FpOperand{xa, ldx, true}, n, d, rows, o, FpEnd::Grad};
            p.x.alpha = scale ? scale + 1 : nullptr;
            products[k++] = p;
        }
        r = fp_gemm(products, k, ws, s);
        if (r) return r;
    }
    return launch_status("linear cross entropy backward");
}

}  // extern "C"
