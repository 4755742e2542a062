// Linear layer on 16-bit floats with its epilogue fused, and its backward pass.
//
//   z = x W^T + bias        y = act(z) + residual
//   dz = dy act'(z)         dx = dz W      dW = dz^T x      dbias = sum over the batch of dz
//
// x [B][IC], W [OC][IC], z, y, dy [B][OC]; products are summed in 32 bits. dz is rounded once
// to the operands' type, because it is an operand of the two products that follow (for 2048 rows
// of 4096 in bf16 dx and dW are off by 0.0024 of their norm, 0.0017 with a dz of 32 bits); dbias sums
// it before that rounding. Products run on the tensor cores (ito_fp_gemm.cu) except for a few
// rows of x, which stream W (ito_fp_rows.cuh). TMA reads operands whose rows start on 16-byte
// boundaries; others are copied into the workspace first, with rows padded to 32 elements.
#include <algorithm>

#include "ito_fp_rows.cuh"

namespace ito {

// Rows of x this kernel takes: 16, and 32 up to 2^24 elements of W. us against the tensor cores'
// kernel's: 4096 x 4096 with 32 rows 12.4 : 14.0, 1024 x 1000 4.3 : 6.9, 8192 x 8192 49 : 36 (the
// blocks' reads of x, which grow with both, pass through L2).
// 4096 x 4096, W from memory (a graph of 16 products with 16 W): 8.7 us with one row, 11.3 with 16,
// 15.6 with 32, at the memory's rate 5.0; with W in L2 6.2, 8.8 and 13.1. 8192 x 8192, beyond L2: 26 with
// one row, 36 with 16 (20). With each step's loads waiting for the step before, one row took 7.4 instead
// of 5.6 with W in L2.
bool fp_rows_kernel(int B, int IC, int OC)
{
    return B <= 16 || (B <= 32 && (int64_t)IC * OC <= (1 << 24));
}

// us of this kernel : the tensor cores'. Classes (Loss) 4096 -> 131072 with 8 rows 162 : 270, 9 207 : 248, 16
// 239 : 174, 32 366 : 175; 1024 -> 50000 with 9 rows 31 : 33, 16 34 : 34, 32 48 : 34. Gated 4096 -> 8192 with 8
// rows 23 : 39, 9 28 : 37, 16 30 : 26; 1024 -> 2048 with 16 rows 4.2 : 7.7, 32 6.8 : 7.8. Of unaligned rows 31,
// 2530 -> 1440, 24 : 11 and a copy of 5.
bool fp_few_rows(int B, int IC, int OC, bool vec)
{
    return B < 16 || (vec && B <= 32 && (int64_t)IC * OC <= (1 << 22));
}

// Logits, forward and in the gradient alike (its logits have to be the same sums). us forward + both gradients, so : in tiles:
// 24 rows 1024 -> 1000 7.7 + 16.3 : 9.6 + 19.0, 2048 -> 2000 10.0 + 25.4 : 13.7 + 28.0, 512 -> 8000 8.6 + 21.4 : 8.8 + 21.4, 256
// -> 16000 11.1 + 24.8 : 8.0 + 22.5, 64 -> 8000 8.8 + 17.3 : 6.2 + 15.0, 4096 -> 1000 13.8 + 25.6 : 10.3 + 21.3; 32 rows 1024
// -> 1000 8.5 + 16.7 : 9.6 + 19.0, 2048 -> 500 11.1 + 17.4 : 9.3 + 16.1, 32768 -> 100 94 + 114 : 17 + 26.
bool fp_few_logits(int B, int IC, int OC, bool vec)
{
    return fp_few_rows(B, IC, OC, vec) && (B <= 16 || (IC >= 512 && IC <= 2048));
}

// --------------------------------------------------------- element-wise passes

// Eight elements to a thread, which start at any element of their row and go to an aligned place (Eight16).
constexpr int kCopyAhead = 2;        // eights of a thread whose loads are in flight together
constexpr int kCopyThreads = 256;

__global__ void __launch_bounds__(kCopyThreads, 6) k_fp_align(const __grid_constant__ FpCopy c)
{
    griddep_wait();
    griddep_launch_dependents();
    const int z = blockIdx.z, rows = c.rows[z], cols = c.cols[z];
    const Divider by = c.by[z];
    const int64_t ld = c.ld[z], ldd = c.ldd[z], total = (int64_t)rows * by.d;
    constexpr int PER = kCopyThreads * kCopyAhead;
    for (int64_t first = (int64_t)blockIdx.x * PER; first < total; first += (int64_t)gridDim.x * PER) {
        const int64_t row0 = first / by.d;               // (one long division a block; what is left fits 32 bits)
        const uint32_t rest = (uint32_t)(first - row0 * by.d), left = (uint32_t)min((int64_t)PER, total - first);
        const uint16_t* const src = c.src[z] + row0 * ld;
        uint16_t* const dst = c.dst[z] + row0 * ldd;
        if (fp_copy_inner(row0, row0 + by(rest + PER - 1), rows, cols, ld)) {
            Eight16 e[kCopyAhead];
            const uint16_t* at[kCopyAhead];
            uint16_t* to[kCopyAhead];
#pragma unroll
            for (int u = 0; u < kCopyAhead; ++u) {
                const uint32_t k = rest + u * kCopyThreads + threadIdx.x, r = by(k), i = (k - r * by.d) * 8;
                at[u] = src + (r * ld + i);
                to[u] = dst + (r * ldd + i);
                e[u].load(at[u]);
            }
            // (what follows a row's end in its padding is never read)
#pragma unroll
            for (int u = 0; u < kCopyAhead; ++u) *reinterpret_cast<uint4*>(to[u]) = e[u].get(at[u]);
            continue;
        }
        for (uint32_t k = rest + threadIdx.x; k < rest + left; k += kCopyThreads) {
            const uint32_t r = by(k);
            const int i = (int)(k - r * by.d) * 8;
            uint16_t x[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = i + q < cols ? src[r * ld + i + q] : 0;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (i + q < cols) dst[r * ldd + i + q] = x[q];
        }
    }
}

// dz = dy act'(z), rounded to the operands' type (dz may be null), and the columns' sums before
// that rounding (dbias may be null). A block takes 64 columns, eight lanes of a warp to a row,
// and a share of the batch; with dbias the shares of the same columns are a cluster, whose first
// block adds their sums in order out of the others' shared memory. So the bias gradient takes no second
// kernel, which at batch 2048 took 5 us before the products could start.
constexpr int kDzColumns = 64;
constexpr int kDzThreads = 256, kDzRows = kDzThreads / 8;    // rows at a time
constexpr int kDzCluster = 8;

template <int ACT>
__global__ void __launch_bounds__(kDzThreads, 1024 / kDzThreads)
    k_fp_dz(const uint16_t* __restrict__ dy, int64_t lddy, const uint16_t* __restrict__ z, int64_t ldz, int type,
            int B, int OC, int shares, int vec, uint16_t* __restrict__ dz, int64_t lddz, float* __restrict__ dbias)
{
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float sums[kDzRows][kDzColumns];
    __shared__ float total[kDzColumns];
    const int row = threadIdx.x >> 3, lane = threadIdx.x & 7;
    const int share = blockIdx.x % shares;     // (its place in the cluster, where there is one)
    const int rows_per = (B + shares - 1) / shares;
    const int c0 = (blockIdx.x / shares) * kDzColumns + lane * 8;
    const int r1 = min(B, (share + 1) * rows_per);
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
    if (c0 < OC) {
        constexpr int U = 4;             // rows whose loads are in flight together
        for (int r0 = share * rows_per + row; r0 < r1; r0 += kDzRows * U) {
            uint4 d[U], q[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = r0 + kDzRows * u;
                d[u] = q[u] = make_uint4(0u, 0u, 0u, 0u);
                if (r < r1) {
                    d[u] = load_eight(dy + r * lddy, c0, OC, vec);
                    if (ACT != ITO_ACT_NONE) q[u] = load_eight(z + r * ldz, c0, OC, vec);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = r0 + kDzRows * u;
                if (r >= r1) break;
                const uint32_t dw[4] = {d[u].x, d[u].y, d[u].z, d[u].w}, qw[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float2 v = unpack16(type, dw[i]);
                    if (ACT != ITO_ACT_NONE) {
                        v = __fmul2_rn(v, act_slope<ACT>(unpack16(type, qw[i])));
                    }
                    s[2 * i] += v.x;
                    s[2 * i + 1] += v.y;
                    o[i] = pack16(type, v.x, v.y);
                }
                // dz's rows are padded to 8 elements: a whole vector always fits
                if (dz) *reinterpret_cast<uint4*>(dz + r * lddz + c0) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
    if (!dbias) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[row][lane * 8 + i] = s[i];
    __syncthreads();
    const int c = threadIdx.x;
    if (c < kDzColumns) {
        float v = 0.0f;
#pragma unroll 32
        for (int w = 0; w < kDzRows; ++w) v += sums[w][c];
        total[c] = v;
    }
    if (shares > 1) cluster_sync();
    const int column = (blockIdx.x / shares) * kDzColumns + c;
    if (share == 0 && c < kDzColumns && column < OC) {
        float v = total[c];
        for (int p = 1; p < shares; ++p) {
            float o;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o) : "r"(mapa_shared(smem_u32(&total[c]), p)) : "memory");
            v += o;
        }
        dbias[column] = v;
    }
    if (shares > 1) cluster_sync();      // the first block has read the others' shared memory
}

// ------------------------------------------------------------------------ host

// shares of the batch: of at least 64 rows each, as many as a cluster has blocks
static int dz_shares(int B)
{
    int n = 1;
    while (n < kDzCluster && B >= 128 * n) n *= 2;
    return n;
}

template <int ACT>
static int run_dz(const void* dy, int64_t lddy, const void* z, int64_t ldz, int type, int B, int OC, int vec,
                  uint16_t* dz, int64_t lddz, float* dbias, cudaStream_t s)
{
    const int shares = dbias ? dz_shares(B) : (B + 63) / 64;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((OC + kDzColumns - 1) / kDzColumns) * shares);
    cfg.blockDim = dim3(kDzThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = shares;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = dbias && shares > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_fp_dz<ACT>, static_cast<const uint16_t*>(dy), lddy,
                                             static_cast<const uint16_t*>(z), ldz, type, B, OC, shares, vec, dz, lddz,
                                             dbias);
    return e == cudaSuccess ? ITO_OK : set_error(ITO_ERR_CUDA, "linear backward launch: %s", cudaGetErrorString(e));
}

int64_t fp_row_stride(int64_t ld, int rows, int cols) { return rows == 1 ? pad8(cols) : ld; }

bool fp_tma_rows(const void* p, int64_t ld, int rows, int cols)
{
    return aligned_to(p, 16) && fp_row_stride(ld, rows, cols) % 8 == 0;
}

// A copy's rows are padded to 64 bytes: rows of 16-byte multiples have TMA read, and the copy write, a sector
// of each 128 bytes more.
static int64_t copy_ld(int64_t cols) { return (cols + 31) & ~int64_t(31); }

bool fp_rows_vec(const void* x, int64_t ldx, const void* W, int64_t ldw, int B, int IC, int OC)
{
    return IC % 8 == 0 && fp_tma_rows(x, ldx, B, IC) && fp_tma_rows(W, ldw, OC, IC);
}

size_t fp_copy_bytes(const void* p, int64_t ld, int rows, int cols)
{
    return fp_tma_rows(p, ld, rows, cols) ? 0 : align256((size_t)rows * copy_ld(cols) * 2);
}

const void* fp_aligned_operand(const void* p, int64_t* ld, int rows, int cols, char** ws, FpCopy* c)
{
    if (fp_tma_rows(p, *ld, rows, cols)) {
        *ld = fp_row_stride(*ld, rows, cols);
        return p;
    }
    uint16_t* dst = reinterpret_cast<uint16_t*>(*ws);
    *ws += fp_copy_bytes(p, *ld, rows, cols);
    c->src[c->n] = static_cast<const uint16_t*>(p);
    c->dst[c->n] = dst;
    c->ld[c->n] = *ld;
    c->ldd[c->n] = copy_ld(cols);
    c->rows[c->n] = rows;
    c->cols[c->n] = cols;
    c->by[c->n] = Divider((cols + 7) / 8);
    ++c->n;
    *ld = copy_ld(cols);
    return dst;
}

int fp_run_copies(const FpCopy& c, cudaStream_t s)
{
    if (!c.n) return ITO_OK;
    int64_t most = 0;
    for (int i = 0; i < c.n; ++i) most = std::max(most, (int64_t)c.rows[i] * ((c.cols[i] + 7) / 8));
    const int64_t blocks = (most + kCopyThreads * kCopyAhead - 1) / (kCopyThreads * kCopyAhead);
    launch_pdl(k_fp_align, dim3((unsigned)std::min<int64_t>(blocks, 1 << 16), 1, c.n), kCopyThreads, 0, s, c);
    return launch_status("linear operand copy");
}

int fp_check_sizes(int B, int IC, int OC)
{
    if (B < 1 || IC < 1 || OC < 1) return set_error(ITO_ERR_SHAPE, "sizes must be >= 1");
    if (B > (1 << 20) || IC > (1 << 20) || OC > (1 << 20)) return set_error(ITO_ERR_SHAPE, "a size above 2^20");
    return ITO_OK;
}

int fp_check_tensor(const void* p, int type, int64_t ld, int rows, int cols, const char* name)
{
    if (!aligned_to(p, type_bytes(type))) return set_error(ITO_ERR_ARG, "%s: misaligned pointer", name);
    if (rows > 1 && ld < cols) return set_error(ITO_ERR_SHAPE, "%s: row stride below its columns", name);
    return ITO_OK;
}

int fp_check_types(int type, int out_type, int act)
{
    if (type != ITO_BF16 && type != ITO_F16) return set_error(ITO_ERR_ARG, "type must be ITO_BF16 or ITO_F16");
    if (out_type != type && out_type != ITO_F32) return set_error(ITO_ERR_ARG, "out_type must be type or ITO_F32");
    if (act < ITO_ACT_NONE || act > ITO_ACT_SILU) return set_error(ITO_ERR_ARG, "unknown activation");
    return ITO_OK;
}

int fp_check_ws(const void* ws, size_t bytes, size_t need)
{
    if (!need) return ITO_OK;
    if (!ws) return set_error(ITO_ERR_ARG, "workspace is NULL");
    if (!aligned_to(ws, 256)) return set_error(ITO_ERR_ARG, "workspace not 256-byte aligned");
    if (bytes < need) return set_error(ITO_ERR_ARG, "workspace too small");
    return ITO_OK;
}

}  // namespace ito

using namespace ito;

extern "C" {

size_t ito_fp_linear_fwd_workspace_size(const void* x, int64_t ldx, const void* W, int64_t ldw, int B, int IC, int OC)
{
    if (fp_check_sizes(B, IC, OC) || fp_rows_kernel(B, IC, OC)) return 0;
    return fp_copy_bytes(x, ldx, B, IC) + fp_copy_bytes(W, ldw, OC, IC) + fp_gemm_ws_bytes(B, OC, IC, false);
}

int ito_fp_linear_fwd(const void* x, int64_t ldx, const void* W, int64_t ldw, const void* bias, const void* residual,
                      int64_t ldr, int type, int out_type, int bias_type, int act, int B, int IC, int OC,
                      void* workspace, size_t workspace_bytes, void* z, int64_t ldz, void* y, int64_t ldy,
                      void* stream)
{
    if (!x || !W || !y) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    int r = fp_check_types(type, out_type, act);
    if (!r) r = fp_check_sizes(B, IC, OC);
    if (r) return r;
    if (bias && bias_type != type && bias_type != ITO_F32)
        return set_error(ITO_ERR_ARG, "bias_type must be type or ITO_F32");
    r = fp_check_tensor(x, type, ldx, B, IC, "x");
    if (!r) r = fp_check_tensor(W, type, ldw, OC, IC, "W");
    if (!r && bias) r = fp_check_tensor(bias, bias_type, OC, 1, OC, "bias");
    if (!r && residual) r = fp_check_tensor(residual, out_type, ldr, B, OC, "residual");
    if (!r && z) r = fp_check_tensor(z, type, ldz, B, OC, "z");
    if (!r) r = fp_check_tensor(y, out_type, ldy, B, OC, "y");
    if (!r) r = fp_check_ws(workspace, workspace_bytes, ito_fp_linear_fwd_workspace_size(x, ldx, W, ldw, B, IC, OC));
    if (r) return r;
    const FpEpilogue e{bias, bias_type, act, residual, ldr, type, out_type, y, ldy, z, ldz};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (fp_rows_kernel(B, IC, OC))
        return fp_run_rows<FpEnd::Linear>(x, ldx, W, ldw, nullptr, 0, B, IC, OC, e, FpMore{}, s);
    char* ws = static_cast<char*>(workspace);
    FpCopy copies{};
    const void* xa = fp_aligned_operand(x, &ldx, B, IC, &ws, &copies);
    const void* wa = fp_aligned_operand(W, &ldw, OC, IC, &ws, &copies);
    r = fp_run_copies(copies, s);
    if (r) return r;
    const FpProduct product{FpOperand{xa, ldx, false}, FpOperand{wa, ldw, false}, B, OC, IC, e, FpEnd::Linear};
    return fp_gemm(&product, 1, ws, s);
}

size_t ito_fp_linear_bwd_workspace_size(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* W,
                                        int64_t ldw, int act, int B, int IC, int OC)
{
    if (fp_check_sizes(B, IC, OC)) return 0;
    const bool dz = act != ITO_ACT_NONE || !fp_tma_rows(dy, lddy, B, OC);
    return (dz ? align256((size_t)B * pad8(OC) * 2) : 0) + fp_copy_bytes(x, ldx, B, IC) + fp_copy_bytes(W, ldw, OC, IC) +
           fp_gemm_ws_bytes(B, IC, OC, true) + fp_gemm_ws_bytes(OC, IC, B, true);
}

int ito_fp_linear_bwd(const void* dy, int64_t lddy, const void* z, int64_t ldz, const void* x, int64_t ldx,
                      const void* W, int64_t ldw, int type, int out_type, int act, int B, int IC, int OC,
                      void* workspace, size_t workspace_bytes, void* dx, int64_t lddx, void* dW, int64_t lddw,
                      float* dbias, void* stream)
{
    if (!dy || (dW && !x) || (dx && !W)) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    if (!dx && !dW && !dbias) return set_error(ITO_ERR_ARG, "no output");
    int r = fp_check_types(type, out_type, act);
    if (!r) r = fp_check_sizes(B, IC, OC);
    if (r) return r;
    if (act != ITO_ACT_NONE && !z) return set_error(ITO_ERR_ARG, "an activation's gradient needs z");
    r = fp_check_tensor(dy, type, lddy, B, OC, "dy");
    if (!r && act != ITO_ACT_NONE) r = fp_check_tensor(z, type, ldz, B, OC, "z");
    if (!r && dW) r = fp_check_tensor(x, type, ldx, B, IC, "x");
    if (!r && dx) r = fp_check_tensor(W, type, ldw, OC, IC, "W");
    if (!r && dx) r = fp_check_tensor(dx, type, lddx, B, IC, "dx");
    if (!r && dW) r = fp_check_tensor(dW, out_type, lddw, OC, IC, "dW");
    if (!r && !aligned_to(dbias, 4)) r = set_error(ITO_ERR_ARG, "dbias: misaligned pointer");
    if (!r)
        r = fp_check_ws(workspace, workspace_bytes,
                        ito_fp_linear_bwd_workspace_size(dy, lddy, x, ldx, W, ldw, act, B, IC, OC));
    if (r) return r;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    // dz is dy itself where nothing changes it and TMA can read it
    const bool own_dz = act != ITO_ACT_NONE || !fp_tma_rows(dy, lddy, B, OC);
    uint16_t* dz = nullptr;
    if (own_dz) {
        dz = reinterpret_cast<uint16_t*>(ws);
        ws += align256((size_t)B * pad8(OC) * 2);
    }
    if (dbias || (own_dz && (dx || dW))) {
        const int vec = fp_tma_rows(dy, lddy, B, OC) && (act == ITO_ACT_NONE || fp_tma_rows(z, ldz, B, OC));
        uint16_t* out = dx || dW ? dz : nullptr;
        switch (act) {
        case ITO_ACT_RELU: r = run_dz<ITO_ACT_RELU>(dy, lddy, z, ldz, type, B, OC, vec, out, pad8(OC), dbias, s); break;
        case ITO_ACT_GELU: r = run_dz<ITO_ACT_GELU>(dy, lddy, z, ldz, type, B, OC, vec, out, pad8(OC), dbias, s); break;
        case ITO_ACT_GELU_TANH:
            r = run_dz<ITO_ACT_GELU_TANH>(dy, lddy, z, ldz, type, B, OC, vec, out, pad8(OC), dbias, s);
            break;
        case ITO_ACT_SILU: r = run_dz<ITO_ACT_SILU>(dy, lddy, z, ldz, type, B, OC, vec, out, pad8(OC), dbias, s); break;
        default: r = run_dz<ITO_ACT_NONE>(dy, lddy, z, ldz, type, B, OC, vec, out, pad8(OC), dbias, s); break;
        }
        if (r) return r;
    }
    const void* d = own_dz ? dz : dy;
    const int64_t ldd = own_dz ? pad8(OC) : fp_row_stride(lddy, B, OC);
    // copies of x and W keep their places in the workspace whether or not both are made
    char* wx = ws;
    char* ww = wx + fp_copy_bytes(x, ldx, B, IC);
    char* wp = ww + fp_copy_bytes(W, ldw, OC, IC);
    FpProduct products[2];
    FpCopy copies{};
    int n = 0;
    if (dx) {
        const void* wa = fp_aligned_operand(W, &ldw, OC, IC, &ww, &copies);
        FpEpilogue e{};
        e.type = e.out_type = type;
        e.y = dx;
        e.ldy = lddx;
        products[n++] = FpProduct{FpOperand{d, ldd, false}, FpOperand{wa, ldw, true}, B, IC, OC, e, FpEnd::Linear};
    }
    if (dW) {
        const void* xa = fp_aligned_operand(x, &ldx, B, IC, &wx, &copies);
        FpEpilogue e{};
        e.type = type;
        e.out_type = out_type;
        e.y = dW;
        e.ldy = lddw;
        products[n++] = FpProduct{FpOperand{d, ldd, true}, FpOperand{xa, ldx, true}, OC, IC, B, e, FpEnd::Linear};
    }
    r = fp_run_copies(copies, s);
    if (!r && n) r = fp_gemm(products, n, wp, s);
    return r ? r : launch_status("linear backward");
}

}  // extern "C"
