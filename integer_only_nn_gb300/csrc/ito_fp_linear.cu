// Linear layer on 16-bit floats with its epilogue fused, and its backward pass.
//
//   z = x W^T + bias        y = act(z) + residual
//   dz = dy act'(z)         dx = dz W      dW = dz^T x      dbias = sum over the batch of dz
//
// x [B][IC], W [OC][IC], z, y, dy [B][OC]; products are summed in 32 bits. dz is rounded once
// to the operands' type, because it is an operand of the two products that follow (for 2048 rows
// of 4096 in bf16 dx and dW are off by 0.0024 of their norm, 0.0017 with a dz of 32 bits); dbias sums
// it before that rounding. Products run on the tensor cores (ito_fp_gemm.cu) except for a few
// rows of x, which stream W (k_fp_rows below). TMA reads operands whose rows start on 16-byte
// boundaries; others are copied into the workspace first, with rows padded to 8 elements.
#include <algorithm>

#include "ito_fp_epilogue.cuh"

namespace ito {

// ------------------------------------------------------------- a few rows of x
//
// With a few rows the product reads W once and does little with it: W's bytes bound it.
// A warp takes 16 rows of W as the 16 x 16 operand of mma.sync and eight rows of x (a token
// each; missing ones are 0) as the 16 x 8 one. The sum over k may be taken in any order, so
// the fragments' k are assigned such that each lane reads 16 consecutive bytes of a row of W
// (k0 + 8 t .. + 7 for lane t of a quad) and the same k of its row of x: two products of
// 16 k from one wide load each. A block's warps share the 16 rows and take turns along k; their
// sums meet in shared memory, in the warps' order.

// Rows of x this kernel takes: 16, and 32 up to 2^24 elements of W. us against the tensor cores'
// kernel's: 4096 x 4096 with 32 rows 12.4 : 14.0, 1024 x 1000 4.3 : 6.9, 8192 x 8192 49 : 36 (the
// blocks' reads of x, which grow with both, pass through L2).
// 4096 x 4096, W from memory (a graph of 16 products with 16 W): 8.7 us with one row, 11.3 with 16,
// 15.6 with 32, at the memory's rate 5.0; with W in L2 6.2, 8.8 and 13.1. 8192 x 8192, beyond L2: 26 with
// one row, 36 with 16 (20). With each step's loads waiting for the step before, one row took 7.4 instead
// of 5.6 with W in L2.
static bool rows_kernel(int B, int IC, int OC)
{
    return B <= 16 || (B <= 32 && (int64_t)IC * OC <= (1 << 24));
}

__device__ __forceinline__ void mma_16816(int type, float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    if (type == ITO_BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// elements k .. k + 7 of a row of n (0 beyond it)
__device__ __forceinline__ uint4 load_eight(const uint16_t* row, int k, int n, bool vec)
{
    if (vec && k + 8 <= n) return __ldg(reinterpret_cast<const uint4*>(row + k));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < n) w[i >> 1] |= (uint32_t)__ldg(row + k + i) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 load_once(const uint16_t* p)      // (read by one block: not for L1)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

constexpr int kRowsSteps = 4;        // steps of 32 k whose loads of W are in flight together
constexpr int kRowsWarps = 8;        // of a block, at most

// VEC: both operands' rows start on 16-byte boundaries and IC is a multiple of 8
template <int NT, bool VEC>
__global__ void __launch_bounds__(kRowsWarps * 32)
    k_fp_rows(const uint16_t* __restrict__ x, int64_t ldx, const uint16_t* __restrict__ W, int64_t ldw, int B, int IC,
              int OC, const __grid_constant__ FpEpilogue e)
{
    constexpr int U = kRowsSteps;
    __shared__ float part[kRowsWarps][16 * 8 * NT];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int warps = blockDim.x >> 5;
    const int oc0 = blockIdx.x * 16;
    const bool in0 = oc0 + g < OC, in1 = oc0 + g + 8 < OC;
    const uint16_t* w0 = W + (int64_t)(in0 ? oc0 + g : 0) * ldw;
    const uint16_t* w1 = W + (int64_t)(in1 ? oc0 + g + 8 : 0) * ldw;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    auto load = [&](const uint16_t* row, int k, bool in) {
        if (VEC) return in && k < IC ? load_once(row + k) : zero;
        return in && k < IC ? load_eight(row, k, IC, false) : zero;
    };
    float c[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[n][i] = 0.0f;
    uint4 a[U], b[U];
    const int stride = warps * U * 32;
    int k0 = warp * U * 32;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        a[u] = load(w0, k0 + u * 32 + t * 8, in0);
        b[u] = load(w1, k0 + u * 32 + t * 8, in1);
    }
    for (; k0 < IC; k0 += stride) {
        // the next steps' rows of W are on their way while these are multiplied
        uint4 an[U], bn[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            an[u] = load(w0, k0 + stride + u * 32 + t * 8, in0);
            bn[u] = load(w1, k0 + stride + u * 32 + t * 8, in1);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool in = n * 8 + g < B;
            const uint16_t* xr = x + (int64_t)(in ? n * 8 + g : 0) * ldx;
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * 32 + t * 8;
                v[u] = in && k < IC ? load_eight(xr, k, IC, VEC) : zero;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                mma_16816(e.type, c[n], a[u].x, b[u].x, a[u].y, b[u].y, v[u].x, v[u].y);
                mma_16816(e.type, c[n], a[u].z, b[u].z, a[u].w, b[u].w, v[u].z, v[u].w);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[u] = an[u];
            b[u] = bn[u];
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[warp][(n * 8 + 2 * t + (i & 1)) * 16 + g + 8 * (i >> 1)] = c[n][i];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * 8 * NT; i += blockDim.x) {
        const int b = i >> 4, oc = oc0 + (i & 15);
        if (b >= B || oc >= OC) continue;
        float s = part[0][i];
        for (int w = 1; w < warps; ++w) s += part[w][i];
        fp_finish(e, b, oc, s);
    }
}

// --------------------------------------------------------- element-wise passes

// Rows whose starts TMA cannot address, copied to rows padded to 8 elements; up to two tensors
// (blockIdx.z).
struct FpCopy {
    const uint16_t* src[2];
    uint16_t* dst[2];
    int64_t ld[2], ldd[2];
    int rows[2], cols[2];
    int n;
};

__global__ void __launch_bounds__(256) k_fp_align(const __grid_constant__ FpCopy c)
{
    griddep_wait();
    griddep_launch_dependents();
    const int z = blockIdx.z;
    const uint16_t* src = c.src[z];
    uint16_t* dst = c.dst[z];
    const int end = min(c.cols[z], ((int)blockIdx.x + 1) * 1024);
    for (int64_t r = blockIdx.y; r < c.rows[z]; r += gridDim.y)
#pragma unroll 4
        for (int i = blockIdx.x * 1024 + threadIdx.x; i < end; i += 256) dst[r * c.ldd[z] + i] = src[r * c.ld[z] + i];
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

static size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// A row's stride says nothing about a single row.
static int64_t row_stride(int64_t ld, int rows, int cols) { return rows == 1 ? pad8(cols) : ld; }

static bool tma_rows(const void* p, int64_t ld, int rows, int cols)
{
    return aligned_to(p, 16) && row_stride(ld, rows, cols) % 8 == 0;
}

static size_t copy_bytes(const void* p, int64_t ld, int rows, int cols)
{
    return tma_rows(p, ld, rows, cols) ? 0 : align256((size_t)rows * pad8(cols) * 2);
}

// The operand itself, or where its aligned copy will be (at *ws, which moves on), noted in `c`.
static const void* aligned_operand(const void* p, int64_t* ld, int rows, int cols, char** ws, FpCopy* c)
{
    if (tma_rows(p, *ld, rows, cols)) {
        *ld = row_stride(*ld, rows, cols);
        return p;
    }
    uint16_t* dst = reinterpret_cast<uint16_t*>(*ws);
    *ws += copy_bytes(p, *ld, rows, cols);
    c->src[c->n] = static_cast<const uint16_t*>(p);
    c->dst[c->n] = dst;
    c->ld[c->n] = *ld;
    c->ldd[c->n] = pad8(cols);
    c->rows[c->n] = rows;
    c->cols[c->n] = cols;
    ++c->n;
    *ld = pad8(cols);
    return dst;
}

static int run_copies(const FpCopy& c, cudaStream_t s)
{
    if (!c.n) return ITO_OK;
    int rows = 0, cols = 0;
    for (int i = 0; i < c.n; ++i) {
        rows = std::max(rows, c.rows[i]);
        cols = std::max(cols, c.cols[i]);
    }
    launch_pdl(k_fp_align, dim3((cols + 1023) / 1024, std::min(rows, 16384), c.n), 256, 0, s, c);
    return launch_status("linear operand copy");
}

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

template <int NT>
static int run_rows(const void* x, int64_t ldx, const void* W, int64_t ldw, int B, int IC, int OC,
                    const FpEpilogue& e, cudaStream_t s)
{
    const int warps = std::min(kRowsWarps, std::max(1, (IC + 32 * kRowsSteps - 1) / (32 * kRowsSteps)));
    const bool vec = IC % 8 == 0 && tma_rows(x, ldx, B, IC) && tma_rows(W, ldw, OC, IC);
    launch_pdl(vec ? k_fp_rows<NT, true> : k_fp_rows<NT, false>, (OC + 15) / 16, warps * 32, 0, s,
               static_cast<const uint16_t*>(x), ldx, static_cast<const uint16_t*>(W), ldw, B, IC, OC, e);
    return launch_status("linear");
}

}  // namespace ito

using namespace ito;

extern "C" {

size_t ito_fp_linear_fwd_workspace_size(const void* x, int64_t ldx, const void* W, int64_t ldw, int B, int IC, int OC)
{
    if (check_sizes(B, IC, OC) || rows_kernel(B, IC, OC)) return 0;
    return copy_bytes(x, ldx, B, IC) + copy_bytes(W, ldw, OC, IC) + fp_gemm_ws_bytes(B, OC, IC, false);
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
    const FpEpilogue e{bias, bias_type, act, residual, ldr, type, out_type, y, ldy, z, ldz};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows_kernel(B, IC, OC)) {
        if (B <= 8) return run_rows<1>(x, ldx, W, ldw, B, IC, OC, e, s);
        if (B <= 16) return run_rows<2>(x, ldx, W, ldw, B, IC, OC, e, s);
        if (B <= 24) return run_rows<3>(x, ldx, W, ldw, B, IC, OC, e, s);
        return run_rows<4>(x, ldx, W, ldw, B, IC, OC, e, s);
    }
    char* ws = static_cast<char*>(workspace);
    FpCopy copies{};
    const void* xa = aligned_operand(x, &ldx, B, IC, &ws, &copies);
    const void* wa = aligned_operand(W, &ldw, OC, IC, &ws, &copies);
    r = run_copies(copies, s);
    if (r) return r;
    const FpProduct product{FpOperand{xa, ldx, false}, FpOperand{wa, ldw, false}, B, OC, IC, e};
    return fp_gemm(&product, 1, ws, s);
}

size_t ito_fp_linear_bwd_workspace_size(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* W,
                                        int64_t ldw, int act, int B, int IC, int OC)
{
    if (check_sizes(B, IC, OC)) return 0;
    const bool dz = act != ITO_ACT_NONE || !tma_rows(dy, lddy, B, OC);
    return (dz ? align256((size_t)B * pad8(OC) * 2) : 0) + copy_bytes(x, ldx, B, IC) + copy_bytes(W, ldw, OC, IC) +
           fp_gemm_ws_bytes(B, IC, OC, true) + fp_gemm_ws_bytes(OC, IC, B, true);
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
    char* ws = static_cast<char*>(workspace);
    // dz is dy itself where nothing changes it and TMA can read it
    const bool own_dz = act != ITO_ACT_NONE || !tma_rows(dy, lddy, B, OC);
    uint16_t* dz = nullptr;
    if (own_dz) {
        dz = reinterpret_cast<uint16_t*>(ws);
        ws += align256((size_t)B * pad8(OC) * 2);
    }
    if (dbias || (own_dz && (dx || dW))) {
        const int vec = tma_rows(dy, lddy, B, OC) && (act == ITO_ACT_NONE || tma_rows(z, ldz, B, OC));
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
    const int64_t ldd = own_dz ? pad8(OC) : row_stride(lddy, B, OC);
    // copies of x and W keep their places in the workspace whether or not both are made
    char* wx = ws;
    char* ww = wx + copy_bytes(x, ldx, B, IC);
    char* wp = ww + copy_bytes(W, ldw, OC, IC);
    FpProduct products[2];
    FpCopy copies{};
    int n = 0;
    if (dx) {
        const void* wa = aligned_operand(W, &ldw, OC, IC, &ww, &copies);
        FpEpilogue e{};
        e.type = e.out_type = type;
        e.y = dx;
        e.ldy = lddx;
        products[n++] = FpProduct{FpOperand{d, ldd, false}, FpOperand{wa, ldw, true}, B, IC, OC, e};
    }
    if (dW) {
        const void* xa = aligned_operand(x, &ldx, B, IC, &wx, &copies);
        FpEpilogue e{};
        e.type = type;
        e.out_type = out_type;
        e.y = dW;
        e.ldy = lddw;
        products[n++] = FpProduct{FpOperand{d, ldd, true}, FpOperand{xa, ldx, true}, OC, IC, B, e};
    }
    r = run_copies(copies, s);
    if (!r && n) r = fp_gemm(products, n, wp, s);
    return r ? r : launch_status("linear backward");
}

}  // extern "C"
