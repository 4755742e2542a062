// Gated layer on 16-bit floats and its backward pass.
//
//   zg = x Wg^T + bg    zu = x Wu^T + bu    h = act(zg) zu
//   dzg = dh zu act'(zg)    dzu = dh act(zg)
//   dx = dzg Wg + dzu Wu    dWg = dzg^T x    dWu = dzu^T x    dbg, dbu = sums over the batch of dzg, dzu
//
// Forward both products share a tile: its first columns of sums are zg's, its last zu's, of the
// same result columns, so x is read once and neither z has to leave the SM (each CTA of a pair
// stages the rows of one of the two weights). A few rows of x stream both weights (ito_fp_rows.cuh).
//
// Backward dzg and dzu stand side by side in the workspace, [B][2][OC padded to K blocks], rounded
// once to the operands' type: dx is one product over both halves of K, dWg and dWu one of both
// halves of rows, and the two share a launch (ito_fp_gemm.cu, FpEnd::Grad). Of a few rows both stream
// the weights (ito_fp_few_grad.cu).
#include "ito_fp_rows.cuh"

namespace ito {

// dzg, dzu and the columns' sums before the rounding (each sum may be null), laid out as k_fp_dz: a
// block takes 64 columns, eight lanes to a row, and a share of the batch; the shares of the same
// columns are a cluster whose first block adds their sums in order. dz's columns from OC up to the
// half's end get 0.
constexpr int kGdColumns = 64;
constexpr int kGdThreads = 256, kGdRows = kGdThreads / 8;    // rows at a time
constexpr int kGdCluster = 8;

struct GatedDz {
    const uint16_t *dh, *zg, *zu;
    int64_t lddh, ldzg, ldzu;
    int type, B, OC, half, shares, vec;
    uint16_t* dz;            // [B][2 half], may be null
    float *dbg, *dbu;
};

template <int ACT>
__global__ void __launch_bounds__(kGdThreads, 4) k_fp_gated_dz(const __grid_constant__ GatedDz a)
{
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float sums[2][kGdRows][kGdColumns];
    __shared__ float total[2][kGdColumns];
    const int row = threadIdx.x >> 3, lane = threadIdx.x & 7;
    const int share = blockIdx.x % a.shares;     // (its place in the cluster, where there is one)
    const int rows_per = (a.B + a.shares - 1) / a.shares;
    const int c0 = (blockIdx.x / a.shares) * kGdColumns + lane * 8;
    const int r1 = min(a.B, (share + 1) * rows_per);
    const int type = a.type;
    float sg[8], su[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sg[i] = su[i] = 0.0f;
    constexpr int U = 2;                         // rows whose loads are in flight together
    for (int r0 = share * rows_per + row; r0 < r1; r0 += kGdRows * U) {
        uint4 d[U], g[U], q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + kGdRows * u;
            d[u] = g[u] = q[u] = make_uint4(0u, 0u, 0u, 0u);
            if (r < r1) {
                d[u] = load_eight(a.dh + r * a.lddh, c0, a.OC, a.vec);
                g[u] = load_eight(a.zg + r * a.ldzg, c0, a.OC, a.vec);
                q[u] = load_eight(a.zu + r * a.ldzu, c0, a.OC, a.vec);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + kGdRows * u;
            if (r >= r1) break;
            const uint32_t dw[4] = {d[u].x, d[u].y, d[u].z, d[u].w}, gw[4] = {g[u].x, g[u].y, g[u].z, g[u].w},
                           qw[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
            uint32_t og[4], ou[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 dv = unpack16(type, dw[i]), gv = unpack16(type, gw[i]);
                const float2 vu = __fmul2_rn(dv, act_value<ACT>(gv));
                const float2 vg = __fmul2_rn(__fmul2_rn(dv, unpack16(type, qw[i])), act_slope<ACT>(gv));
                sg[2 * i] += vg.x;
                sg[2 * i + 1] += vg.y;
                su[2 * i] += vu.x;
                su[2 * i + 1] += vu.y;
                og[i] = pack16(type, vg.x, vg.y);
                ou[i] = pack16(type, vu.x, vu.y);
            }
            if (a.dz) {
                uint16_t* out = a.dz + r * 2 * a.half + c0;
                *reinterpret_cast<uint4*>(out) = make_uint4(og[0], og[1], og[2], og[3]);
                *reinterpret_cast<uint4*>(out + a.half) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
            }
        }
    }
    if (!a.dbg && !a.dbu) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        sums[0][row][lane * 8 + i] = sg[i];
        sums[1][row][lane * 8 + i] = su[i];
    }
    __syncthreads();
    const int which = threadIdx.x / kGdColumns, c = threadIdx.x % kGdColumns;
    if (which < 2) {
        float v = 0.0f;
#pragma unroll 32
        for (int w = 0; w < kGdRows; ++w) v += sums[which][w][c];
        total[which][c] = v;
    }
    if (a.shares > 1) cluster_sync();
    const int column = (blockIdx.x / a.shares) * kGdColumns + c;
    if (share == 0 && which < 2 && column < a.OC) {
        float v = total[which][c];
        for (int p = 1; p < a.shares; ++p) {
            float o;
            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                         : "=f"(o)
                         : "r"(mapa_shared(smem_u32(&total[which][c]), p))
                         : "memory");
            v += o;
        }
        float* out = which ? a.dbu : a.dbg;
        if (out) out[column] = v;
    }
    if (a.shares > 1) cluster_sync();      // the first block has read the others' shared memory
}

// ------------------------------------------------------------------------ host

static int gated_half(int OC) { return (OC + 63) / 64 * 64; }

// Shares of the batch. With sums they cost a block its barriers: as many as give an SM four blocks, of 64 rows at
// least, and as a cluster has blocks (1262 x 16128, us: 8 shares 47, as many as this 38).
static int gated_shares(int B, int half, bool sums)
{
    if (!sums) return (B + 63) / 64;
    int n = 1;
    while (n < kGdCluster && B >= 128 * n && half / kGdColumns * n < 4 * num_sms()) n *= 2;
    return n;
}

template <int ACT>
static int run_gated_dz(GatedDz a, cudaStream_t s)
{
    const bool sums = a.dbg || a.dbu;
    a.shares = gated_shares(a.B, a.half, sums);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.half / kGdColumns) * a.shares);
    cfg.blockDim = dim3(kGdThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = a.shares;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = sums && a.shares > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_fp_gated_dz<ACT>, a);
    return e == cudaSuccess ? ITO_OK : set_error(ITO_ERR_CUDA, "gated layer backward launch: %s", cudaGetErrorString(e));
}

static bool gated_few(const void* x, int64_t ldx, const void* Wg, int64_t ldwg, const void* Wu, int64_t ldwu, int B, int IC,
                      int OC)
{
    return fp_few_rows(B, IC, OC, fp_rows_vec(x, ldx, Wg, ldwg, B, IC, OC) && fp_tma_rows(Wu, ldwu, OC, IC));
}

static int check_gated(int type, int act, int B, int IC, int OC)
{
    const int r = fp_check_types(type, type, act);
    return r ? r : fp_check_sizes(B, IC, OC);
}

}  // namespace ito

using namespace ito;

extern "C" {

size_t ito_fp_gated_linear_fwd_workspace_size(const void* x, int64_t ldx, const void* Wg, int64_t ldwg, const void* Wu,
                                              int64_t ldwu, int B, int IC, int OC)
{
    if (fp_check_sizes(B, IC, OC) || gated_few(x, ldx, Wg, ldwg, Wu, ldwu, B, IC, OC)) return 0;
    return fp_copy_bytes(x, ldx, B, IC) + fp_copy_bytes(Wg, ldwg, OC, IC) + fp_copy_bytes(Wu, ldwu, OC, IC) +
           fp_gemm_ws_bytes(B, OC, IC, false, FpEnd::Gated);
}

int ito_fp_gated_linear_fwd(const void* x, int64_t ldx, const void* Wg, int64_t ldwg, const void* Wu, int64_t ldwu,
                            const void* bias_g, const void* bias_u, int type, int bias_type, int act, int B, int IC,
                            int OC, void* workspace, size_t workspace_bytes, void* zg, int64_t ldzg, void* zu,
                            int64_t ldzu, void* h, int64_t ldh, void* stream)
{
    if (!x || !Wg || !Wu || !h) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    if (!zg != !zu) return set_error(ITO_ERR_ARG, "zg and zu: both or neither");
    int r = check_gated(type, act, B, IC, OC);
    if (r) return r;
    if ((bias_g || bias_u) && bias_type != type && bias_type != ITO_F32)
        return set_error(ITO_ERR_ARG, "bias_type must be type or ITO_F32");
    r = fp_check_tensor(x, type, ldx, B, IC, "x");
    if (!r) r = fp_check_tensor(Wg, type, ldwg, OC, IC, "Wg");
    if (!r) r = fp_check_tensor(Wu, type, ldwu, OC, IC, "Wu");
    if (!r && bias_g) r = fp_check_tensor(bias_g, bias_type, OC, 1, OC, "bias_g");
    if (!r && bias_u) r = fp_check_tensor(bias_u, bias_type, OC, 1, OC, "bias_u");
    if (!r && zg) r = fp_check_tensor(zg, type, ldzg, B, OC, "zg");
    if (!r && zu) r = fp_check_tensor(zu, type, ldzu, B, OC, "zu");
    if (!r) r = fp_check_tensor(h, type, ldh, B, OC, "h");
    if (!r)
        r = fp_check_ws(workspace, workspace_bytes,
                        ito_fp_gated_linear_fwd_workspace_size(x, ldx, Wg, ldwg, Wu, ldwu, B, IC, OC));
    if (r) return r;
    const FpEpilogue e{bias_g, bias_type, act, nullptr, 0, type, type, h, ldh, zg, ldzg};
    FpMore more{};
    more.bias2 = bias_u;
    more.z2 = zu;
    more.ldz2 = ldzu;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (gated_few(x, ldx, Wg, ldwg, Wu, ldwu, B, IC, OC))
        return fp_run_rows<FpEnd::Gated>(x, ldx, Wg, ldwg, Wu, ldwu, B, IC, OC, e, more, s);
    char* ws = static_cast<char*>(workspace);
    FpCopy copies{};
    const void* xa = fp_aligned_operand(x, &ldx, B, IC, &ws, &copies);
    const void* ga = fp_aligned_operand(Wg, &ldwg, OC, IC, &ws, &copies);
    const void* ua = fp_aligned_operand(Wu, &ldwu, OC, IC, &ws, &copies);
    r = fp_run_copies(copies, s);
    if (r) return r;
    FpProduct p{FpOperand{xa, ldx, false}, FpOperand{ga, ldwg, false}, B, OC, IC, e, FpEnd::Gated, more};
    p.B2 = FpOperand{ua, ldwu, false};
    return fp_gemm(&p, 1, ws, s);
}

size_t ito_fp_gated_linear_bwd_workspace_size(const void* x, int64_t ldx, const void* Wg, int64_t ldwg, const void* Wu,
                                              int64_t ldwu, int B, int IC, int OC)
{
    if (fp_check_sizes(B, IC, OC)) return 0;
    const int half = gated_half(OC);
    if (fp_few_grad_rows(B)) return align256((size_t)B * 2 * half * 2) + fp_few_grad_ws_bytes(B, OC, IC, 2);
    return align256((size_t)B * 2 * half * 2) + fp_copy_bytes(x, ldx, B, IC) + fp_copy_bytes(Wg, ldwg, OC, IC) +
           fp_copy_bytes(Wu, ldwu, OC, IC) + fp_gemm_ws_bytes(B, IC, 2 * half, true, FpEnd::Grad) +
           fp_gemm_ws_bytes(OC, IC, B, true, FpEnd::Grad, 2);
}

int ito_fp_gated_linear_bwd(const void* dh, int64_t lddh, const void* zg, int64_t ldzg, const void* zu, int64_t ldzu,
                            const void* x, int64_t ldx, const void* Wg, int64_t ldwg, const void* Wu, int64_t ldwu,
                            int type, int out_type, int act, int B, int IC, int OC, void* workspace,
                            size_t workspace_bytes, void* dx, int64_t lddx, void* dWg, int64_t lddwg, void* dWu,
                            int64_t lddwu, float* dbias_g, float* dbias_u, void* stream)
{
    if (!dh || !zg || !zu || (dWg && !x) || (dx && (!Wg || !Wu))) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    if (!dWg != !dWu) return set_error(ITO_ERR_ARG, "dWg and dWu: both or neither");
    if (!dx && !dWg && !dbias_g && !dbias_u) return set_error(ITO_ERR_ARG, "no output");
    int r = check_gated(type, act, B, IC, OC);
    if (!r) r = fp_check_types(type, out_type, act);
    if (r) return r;
    r = fp_check_tensor(dh, type, lddh, B, OC, "dh");
    if (!r) r = fp_check_tensor(zg, type, ldzg, B, OC, "zg");
    if (!r) r = fp_check_tensor(zu, type, ldzu, B, OC, "zu");
    if (!r && dWg) r = fp_check_tensor(x, type, ldx, B, IC, "x");
    if (!r && dx) r = fp_check_tensor(Wg, type, ldwg, OC, IC, "Wg");
    if (!r && dx) r = fp_check_tensor(Wu, type, ldwu, OC, IC, "Wu");
    if (!r && dx) r = fp_check_tensor(dx, type, lddx, B, IC, "dx");
    if (!r && dWg) r = fp_check_tensor(dWg, out_type, lddwg, OC, IC, "dWg");
    if (!r && dWu) r = fp_check_tensor(dWu, out_type, lddwu, OC, IC, "dWu");
    if (!r && (!aligned_to(dbias_g, 4) || !aligned_to(dbias_u, 4))) r = set_error(ITO_ERR_ARG, "dbias: misaligned pointer");
    if (!r)
        r = fp_check_ws(workspace, workspace_bytes,
                        ito_fp_gated_linear_bwd_workspace_size(x, ldx, Wg, ldwg, Wu, ldwu, B, IC, OC));
    if (r) return r;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    const int half = gated_half(OC);
    GatedDz a{};
    a.dh = static_cast<const uint16_t*>(dh);
    a.zg = static_cast<const uint16_t*>(zg);
    a.zu = static_cast<const uint16_t*>(zu);
    a.lddh = lddh;
    a.ldzg = ldzg;
    a.ldzu = ldzu;
    a.type = type;
    a.B = B;
    a.OC = OC;
    a.half = half;
    a.vec = fp_tma_rows(dh, lddh, B, OC) && fp_tma_rows(zg, ldzg, B, OC) && fp_tma_rows(zu, ldzu, B, OC);
    a.dz = dx || dWg ? reinterpret_cast<uint16_t*>(ws) : nullptr;
    a.dbg = dbias_g;
    a.dbu = dbias_u;
    switch (act) {
    case ITO_ACT_RELU: r = run_gated_dz<ITO_ACT_RELU>(a, s); break;
    case ITO_ACT_GELU: r = run_gated_dz<ITO_ACT_GELU>(a, s); break;
    case ITO_ACT_GELU_TANH: r = run_gated_dz<ITO_ACT_GELU_TANH>(a, s); break;
    case ITO_ACT_SILU: r = run_gated_dz<ITO_ACT_SILU>(a, s); break;
    default: r = run_gated_dz<ITO_ACT_NONE>(a, s); break;
    }
    if (r) return r;
    if (fp_few_grad_rows(B)) {
        if (!a.dz) return ITO_OK;
        FpFewGrad p{{a.dz, a.dz + half}, 2 * half,
                    {static_cast<const uint16_t*>(Wg), static_cast<const uint16_t*>(Wu)}, {ldwg, ldwu},
                    static_cast<const uint16_t*>(x), ldx, type, out_type, B, OC, IC, nullptr, dx, lddx, {dWg, dWu},
                    {lddwg, lddwu}};
        return fp_few_grad(p, ws + align256((size_t)B * 2 * half * 2), s);
    }
    // the copies keep their places in the workspace whether or not all are made
    char* wx = ws + align256((size_t)B * 2 * half * 2);
    char* wg = wx + fp_copy_bytes(x, ldx, B, IC);
    char* wu = wg + fp_copy_bytes(Wg, ldwg, OC, IC);
    char* wp = wu + fp_copy_bytes(Wu, ldwu, OC, IC);
    FpProduct products[2];
    FpCopy copies{};
    int n = 0;
    if (dx) {
        const void* ga = fp_aligned_operand(Wg, &ldwg, OC, IC, &wg, &copies);
        const void* ua = fp_aligned_operand(Wu, &ldwu, OC, IC, &wu, &copies);
        FpEpilogue e{};
        e.type = e.out_type = type;
        e.y = dx;
        e.ldy = lddx;
        FpProduct p{FpOperand{a.dz, 2 * half, false}, FpOperand{ga, ldwg, true}, B, IC, 2 * half, e, FpEnd::Grad};
        p.B2 = FpOperand{ua, ldwu, true};
        p.k_half = half;
        p.k_rows = OC;
        products[n++] = p;
    }
    if (dWg) {
        const void* xa = fp_aligned_operand(x, &ldx, B, IC, &wx, &copies);
        FpEpilogue e{};
        e.type = type;
        e.out_type = out_type;
        e.y = dWg;
        e.ldy = lddwg;
        FpProduct p{FpOperand{a.dz, 2 * half, true}, FpOperand{xa, ldx, true}, OC, IC, B, e, FpEnd::Grad};
        p.a_half = half;
        p.x.y2 = dWu;
        p.x.ldy2 = lddwu;
        products[n++] = p;
    }
    r = fp_run_copies(copies, s);
    if (!r && n) r = fp_gemm(products, n, wp, s);
    return r ? r : launch_status("gated layer backward");
}

}  // extern "C"
