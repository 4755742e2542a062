// The linear layer's products on the tensor cores: C[m][n] = sum_k A(m, k) B(n, k) for 16-bit
// float operands, summed in 32 bits in tensor memory, with bias, activation, residual and both
// roundings in the epilogue.
//
// Operands come by TMA with 128-byte swizzle, K-major ([rows][K]) or MN-major ([K][rows]), so
// the forward product (x W^T), dx = dz W and dW = dz^T x read the same row-major tensors and
// nothing is transposed. A producer warp keeps the ring of stages full, one thread issues
// tcgen05.mma, and the epilogue warps drain one of two accumulators while the other fills.
//
// Two kernels: a CTA pair works on 256 x 256 tiles (each SM stages half of B, so a byte from L2
// feeds twice the work), for results with enough such tiles to occupy the device; 128 x 128 and
// 128 x 64 tiles of one CTA, with K cut into slices where there are few tiles, for the rest.
// Slices write their sums in 32 bits to the workspace, and a second kernel adds them in a fixed
// order and does the epilogue.
#include <cstring>

#include "ito_fp_epilogue.cuh"

namespace ito {

struct FpTiles {
    int num_m, num_n, group;
    // groups of `group` row tiles sweep all column tiles: neighbours in time share operands in L2
    __device__ __forceinline__ void coords(int t, int& tm, int& tn) const
    {
        const int per_group = group * num_n;
        const int g = t / per_group;
        const int first_m = g * group;
        const int gm = min(group, num_m - first_m);
        const int r = t - g * per_group;
        tm = first_m + r % gm;
        tn = r / gm;
    }
};

// Instruction descriptor, kind::f16 (see idesc_bf16_f32): format 1 = bf16, 0 = f16
__host__ __device__ constexpr uint32_t fp_idesc(int M, int N, bool a_mn, bool b_mn, bool bf16)
{
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

struct FpGemmArgs {
    FpEpilogue e;
    int M, N, K;
    int a_mn, b_mn;
    uint32_t idesc;
    int group;
    int splits, kb_per_split;   // K slices (1: none); slices go to mapS
    int y_tma, z_tma;           // rows of y and z that TMA stores can take
    int r_vec;                  // rows of the residual that 16-byte loads can take
    int* err;
};

// ------------------------------------------------------------------ epilogue
//
// A warp holds 32 rows (its lanes) of 64 columns of sums at a time. Its results go through its
// own 4 KB of shared memory (32 rows of 128 bytes, 16-byte chunk j of row r at j ^ (r % 8), the
// 128-byte swizzle) and leave by TMA, which clips them at the tensor's edges, or, where rows do
// not start on 16-byte boundaries, by coalesced plain stores.

__device__ __forceinline__ void box_begin(int lane)
{
    if (lane == 0) bulk_wait_read_all();
    __syncwarp();
}

__device__ __forceinline__ void box_end_tma(const CUtensorMap* map, const uint8_t* stg, int lane, int col, int row)
{
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(map, stg, col, row);
        bulk_commit();
    }
}

// the staged box by plain stores: a lane takes one 4-byte word of every row
__device__ __forceinline__ void box_end_plain(void* out, bool wide, int64_t ld, const uint8_t* stg, int lane, int col,
                                              int row, int M, int N)
{
    __syncwarp();
    for (int r = 0; r < 32 && row + r < M; ++r) {
        const uint32_t w =
            *reinterpret_cast<const uint32_t*>(stg + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
        if (wide) {
            if (col + lane < N) static_cast<uint32_t*>(out)[(row + r) * ld + col + lane] = w;
        } else {
            uint16_t* dst = static_cast<uint16_t*>(out) + (row + r) * ld + col + 2 * lane;
            if (col + 2 * lane < N) dst[0] = (uint16_t)w;
            if (col + 2 * lane + 1 < N) dst[1] = (uint16_t)(w >> 16);
        }
    }
    __syncwarp();
}

__device__ __forceinline__ void box16(const float (&v)[64], int type, const CUtensorMap* map, bool tma, void* out,
                                      int64_t ld, uint8_t* stg, int lane, int col, int row, int M, int N)
{
    box_begin(lane);
    const uint32_t at = smem_u32(stg) + lane * 128;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        st_shared_v4(at + ((j ^ (lane & 7)) << 4), (int)pack16(type, v[8 * j], v[8 * j + 1]),
                     (int)pack16(type, v[8 * j + 2], v[8 * j + 3]), (int)pack16(type, v[8 * j + 4], v[8 * j + 5]),
                     (int)pack16(type, v[8 * j + 6], v[8 * j + 7]));
    if (tma) box_end_tma(map, stg, lane, col, row);
    else box_end_plain(out, false, ld, stg, lane, col, row, M, N);
}

// 64 columns in 32 bits are two boxes
__device__ __forceinline__ void stage32(const float (&v)[64], int h, uint8_t* stg, int lane)
{
    box_begin(lane);
    const uint32_t at = smem_u32(stg) + lane * 128;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int i = 32 * h + 4 * j;
        st_shared_v4(at + ((j ^ (lane & 7)) << 4), __float_as_int(v[i]), __float_as_int(v[i + 1]),
                     __float_as_int(v[i + 2]), __float_as_int(v[i + 3]));
    }
}

template <int ACT>
__device__ __forceinline__ void activate(float (&v)[64])
{
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = act_value(ACT, v[i]);
}

__device__ __forceinline__ void finish_group(const FpGemmArgs& a, const CUtensorMap* mapY, const CUtensorMap* mapZ,
                                             float (&v)[64], const float* bias, uint8_t* stg, int lane, int col,
                                             int row)
{
    const FpEpilogue& e = a.e;
    if (e.bias) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float4 b = *reinterpret_cast<const float4*>(bias + 4 * j);
            v[4 * j] += b.x;
            v[4 * j + 1] += b.y;
            v[4 * j + 2] += b.z;
            v[4 * j + 3] += b.w;
        }
    }
    if (e.z) box16(v, e.type, mapZ, a.z_tma, e.z, e.ldz, stg, lane, col, row, a.M, a.N);
    switch (e.act) {
    case ITO_ACT_RELU: activate<ITO_ACT_RELU>(v); break;
    case ITO_ACT_GELU: activate<ITO_ACT_GELU>(v); break;
    case ITO_ACT_GELU_TANH: activate<ITO_ACT_GELU_TANH>(v); break;
    case ITO_ACT_SILU: activate<ITO_ACT_SILU>(v); break;
    default: break;
    }
    if (e.residual && row + lane < a.M) {
        if (e.out_type == ITO_F32) {
            const float* r = static_cast<const float*>(e.residual) + (row + lane) * e.ldr + col;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (a.r_vec && col + 4 * j + 4 <= a.N) {
                    const float4 q = *reinterpret_cast<const float4*>(r + 4 * j);
                    v[4 * j] += q.x;
                    v[4 * j + 1] += q.y;
                    v[4 * j + 2] += q.z;
                    v[4 * j + 3] += q.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (col + 4 * j + i < a.N) v[4 * j + i] += r[4 * j + i];
                }
            }
        } else {
            const uint16_t* r = static_cast<const uint16_t*>(e.residual) + (row + lane) * e.ldr + col;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t w[4] = {0u, 0u, 0u, 0u};
                if (a.r_vec && col + 8 * j + 8 <= a.N) {
                    const uint4 q = *reinterpret_cast<const uint4*>(r + 8 * j);
                    w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (col + 8 * j + i < a.N) w[i >> 1] |= (uint32_t)r[8 * j + i] << (16 * (i & 1));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack16(e.out_type, w[i]);
                    v[8 * j + 2 * i] += f.x;
                    v[8 * j + 2 * i + 1] += f.y;
                }
            }
        }
    }
    if (e.out_type != ITO_F32) {
        box16(v, e.out_type, mapY, a.y_tma, e.y, e.ldy, stg, lane, col, row, a.M, a.N);
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (col + 32 * h >= a.N) continue;
        stage32(v, h, stg, lane);
        if (a.y_tma) box_end_tma(mapY, stg, lane, col + 32 * h, row);
        else box_end_plain(e.y, true, e.ldy, stg, lane, col + 32 * h, row, a.M, a.N);
    }
}

// this warp's columns of the bias, in 32 bits, into shared memory (0 beyond the edge)
__device__ __forceinline__ void stage_bias(const FpGemmArgs& a, float* bias, int cols, int col, int lane)
{
    if (!a.e.bias) return;
    __syncwarp();
    for (int i = lane; i < cols; i += 32) bias[i] = col + i < a.N ? load_typed(a.e.bias, a.e.bias_type, col + i) : 0.0f;
    __syncwarp();
}

__device__ __forceinline__ void load_sums(uint32_t taddr, float (&v)[64])
{
    uint32_t r[32];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        tmem_ld32(taddr + 32 * h, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[32 * h + i] = __uint_as_float(r[i]);
    }
}

// ----------------------------------------------------------------- one CTA

template <int BN>
struct FpCfg {
    static constexpr int BM = 128, BK = 64;
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int EPI_WARPS = BN / 16;            // 64 columns to a warp
    static constexpr int THREADS = 64 + EPI_WARPS * 32;
    static constexpr int TMEM_COLS = 2 * BN;
    static constexpr int STAGES = BN == 128 ? 5 : 8;
    static constexpr int STAGING_BYTES = EPI_WARPS * (4096 + 256);
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + STAGING_BYTES + 1024 + 256;
};

template <int BN>
__global__ void __launch_bounds__(FpCfg<BN>::THREADS, 1)
    k_fp_gemm(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
              const __grid_constant__ CUtensorMap mapY, const __grid_constant__ CUtensorMap mapZ,
              const __grid_constant__ CUtensorMap mapS, const __grid_constant__ FpGemmArgs a)
{
    using Cfg = FpCfg<BN>;
    constexpr int BM = Cfg::BM, BK = Cfg::BK, STAGES = Cfg::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* staging = smem + STAGES * Cfg::STAGE_BYTES;
    float* biases = reinterpret_cast<float*>(staging + Cfg::EPI_WARPS * 4096);
    uint64_t* full_bar = reinterpret_cast<uint64_t*>(staging + Cfg::STAGING_BYTES);
    uint64_t* empty_bar = full_bar + STAGES;
    uint64_t* accf_bar = empty_bar + STAGES;
    uint64_t* acce_bar = accf_bar + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce_bar + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const FpTiles tiles{(a.M + BM - 1) / BM, (a.N + BN - 1) / BN, a.group};
    const int num_items = tiles.num_m * tiles.num_n * a.splits;
    const int num_kb = (a.K + BK - 1) / BK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf_bar[b], 1);
            mbar_init(&acce_bar[b], Cfg::EPI_WARPS);
        }
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&mapA);
        prefetch_tensormap(&mapB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    griddep_wait();
    griddep_launch_dependents();

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int w = blockIdx.x; ok && w < num_items; w += gridDim.x) {
                int tm, tn;
                tiles.coords(w / a.splits, tm, tn);
                const int lo = (w % a.splits) * a.kb_per_split, hi = min(num_kb, lo + a.kb_per_split);
                for (int kb = lo; kb < hi; ++kb) {
                    if (!mbar_wait(&empty_bar[stage], phase ^ 1, abort_flag, a.err)) { ok = false; break; }
                    mbar_arrive_expect_tx(&full_bar[stage], Cfg::STAGE_BYTES);
                    uint8_t* sA = smem + stage * Cfg::STAGE_BYTES;
                    uint8_t* sB = sA + Cfg::A_BYTES;
                    if (!a.a_mn) {
                        tma_load_2d(&mapA, &full_bar[stage], sA, kb * BK, tm * BM);
                    } else {
                        tma_load_2d(&mapA, &full_bar[stage], sA, tm * BM, kb * BK);
                        tma_load_2d(&mapA, &full_bar[stage], sA + 8192, tm * BM + 64, kb * BK);
                    }
                    if (!a.b_mn) {
                        tma_load_2d(&mapB, &full_bar[stage], sB, kb * BK, tn * BN);
                    } else {
#pragma unroll
                        for (int j = 0; j < BN / 64; ++j)
                            tma_load_2d(&mapB, &full_bar[stage], sB + j * 8192, tn * BN + j * 64, kb * BK);
                    }
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0, buf = 0;
            uint32_t phase = 0, buf_phase = 0;
            bool ok = true;
            // a 16-element K step: 32 bytes inside the swizzled row (K-major), 16 rows of 128 bytes (MN-major)
            const uint32_t a_step = a.a_mn ? 2048 : 32, a_lbo = a.a_mn ? 8192 : 16;
            const uint32_t b_step = a.b_mn ? 2048 : 32, b_lbo = a.b_mn ? 8192 : 16;
            for (int w = blockIdx.x; ok && w < num_items; w += gridDim.x) {
                const int lo = (w % a.splits) * a.kb_per_split, hi = min(num_kb, lo + a.kb_per_split);
                if (!mbar_wait(&acce_bar[buf], buf_phase ^ 1, abort_flag, a.err)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(buf * BN);
                for (int kb = lo; kb < hi; ++kb) {
                    if (!mbar_wait(&full_bar[stage], phase, abort_flag, a.err)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(smem + stage * Cfg::STAGE_BYTES), b0 = a0 + Cfg::A_BYTES;
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k)
                        tc_mma_bf16(d, smem_desc_sw128(a0 + k * a_step, a_lbo, 1024),
                                    smem_desc_sw128(b0 + k * b_step, b_lbo, 1024), a.idesc, (kb > lo || k > 0) ? 1u : 0u);
                    tc_commit(&empty_bar[stage]);
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                tc_commit(&accf_bar[buf]);
                if (++buf == 2) { buf = 0; buf_phase ^= 1; }
            }
        }
    } else {
        const int e = warp - 2, quad = warp & 3, part = e >> 2;
        uint8_t* stg = staging + e * 4096;
        float* bias = biases + e * 64;
        int buf = 0;
        uint32_t buf_phase = 0;
        for (int w = blockIdx.x; w < num_items; w += gridDim.x) {
            int tm, tn;
            tiles.coords(w / a.splits, tm, tn);
            const int row = tm * BM + quad * 32, col = tn * BN + part * 64;
            stage_bias(a, bias, 64, col, lane);
            if (!mbar_wait(&accf_bar[buf], buf_phase, abort_flag, a.err)) break;
            tc_fence_after();
            float v[64];
            load_sums(tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * BN + part * 64), v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acce_bar[buf]);
            if (++buf == 2) { buf = 0; buf_phase ^= 1; }
            if (row >= a.M || col >= a.N) continue;
            if (a.splits > 1) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (col + 32 * h >= a.N) continue;
                    stage32(v, h, stg, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&mapS, stg, col + 32 * h, row, w % a.splits);
                        bulk_commit();
                    }
                }
            } else {
                finish_group(a, &mapY, &mapZ, v, bias, stg, lane, col, row);
            }
        }
        if (lane == 0) bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
    }
}

// ---------------------------------------------------------------- CTA pair

struct FpPairCfg {
    static constexpr int BM = 128, BN = 256, BK = 64;
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = (BN / 2) * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = 5;
    static constexpr int EPI_WARPS = 8;
    static constexpr int THREADS = 64 + EPI_WARPS * 32;
    static constexpr int TMEM_COLS = 512;
    static constexpr int STAGING_BYTES = EPI_WARPS * (4096 + 512);
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + STAGING_BYTES + 1024 + 256;
};

__global__ void __launch_bounds__(FpPairCfg::THREADS, 1)
    k_fp_gemm_pair(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                   const __grid_constant__ CUtensorMap mapY, const __grid_constant__ CUtensorMap mapZ,
                   const __grid_constant__ FpGemmArgs a)
{
    using Cfg = FpPairCfg;
    constexpr int BM = Cfg::BM, BN = Cfg::BN, BK = Cfg::BK, STAGES = Cfg::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* staging = smem + STAGES * Cfg::STAGE_BYTES;
    float* biases = reinterpret_cast<float*>(staging + Cfg::EPI_WARPS * 4096);
    uint64_t* full_bar = reinterpret_cast<uint64_t*>(staging + Cfg::STAGING_BYTES);
    uint64_t* empty_bar = full_bar + STAGES;
    uint64_t* accf_bar = empty_bar + STAGES;
    uint64_t* acce_bar = accf_bar + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce_bar + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
    const FpTiles tiles{(a.M + 2 * BM - 1) / (2 * BM), (a.N + BN - 1) / BN, a.group};
    const int num_tiles = tiles.num_m * tiles.num_n;
    const int num_kb = (a.K + BK - 1) / BK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf_bar[b], 1);
            mbar_init(&acce_bar[b], 2 * Cfg::EPI_WARPS);   // epilogue warps of both CTAs
        }
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&mapA);
        prefetch_tensormap(&mapB);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    griddep_wait();
    griddep_launch_dependents();

    if (warp == 0) {
        // both CTAs load; every load completes on the leader's barrier
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int w = cluster; ok && w < num_tiles; w += nclusters) {
                int tm, tn;
                tiles.coords(w, tm, tn);
                const int rowA = tm * 2 * BM + (int)rank * BM, rowB = tn * BN + (int)rank * (BN / 2);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(&empty_bar[stage], phase ^ 1, abort_flag, a.err)) { ok = false; break; }
                    if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * Cfg::STAGE_BYTES);
                    const uint32_t fb = mapa_shared(smem_u32(&full_bar[stage]), 0);
                    uint8_t* sA = smem + stage * Cfg::STAGE_BYTES;
                    uint8_t* sB = sA + Cfg::A_BYTES;
                    if (!a.a_mn) {
                        tma_load_2d_pair(&mapA, fb, sA, kb * BK, rowA);
                    } else {
                        tma_load_2d_pair(&mapA, fb, sA, rowA, kb * BK);
                        tma_load_2d_pair(&mapA, fb, sA + 8192, rowA + 64, kb * BK);
                    }
                    if (!a.b_mn) {
                        tma_load_2d_pair(&mapB, fb, sB, kb * BK, rowB);
                    } else {
                        tma_load_2d_pair(&mapB, fb, sB, rowB, kb * BK);
                        tma_load_2d_pair(&mapB, fb, sB + 8192, rowB + 64, kb * BK);
                    }
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
            }
        }
    } else if (warp == 1) {
        if (leader && lane == 0) {
            int stage = 0, buf = 0;
            uint32_t phase = 0, buf_phase = 0;
            bool ok = true;
            const uint32_t a_step = a.a_mn ? 2048 : 32, a_lbo = a.a_mn ? 8192 : 16;
            const uint32_t b_step = a.b_mn ? 2048 : 32, b_lbo = a.b_mn ? 8192 : 16;
            for (int w = cluster; ok && w < num_tiles; w += nclusters) {
                if (!mbar_wait(&acce_bar[buf], buf_phase ^ 1, abort_flag, a.err)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(buf * BN);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(&full_bar[stage], phase, abort_flag, a.err)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(smem + stage * Cfg::STAGE_BYTES), b0 = a0 + Cfg::A_BYTES;
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k)
                        tc_mma_bf16_pair(d, smem_desc_sw128(a0 + k * a_step, a_lbo, 1024),
                                         smem_desc_sw128(b0 + k * b_step, b_lbo, 1024), a.idesc,
                                         (kb > 0 || k > 0) ? 1u : 0u);
                    tc_commit_pair_mc(&empty_bar[stage], 0x3);
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                tc_commit_pair_mc(&accf_bar[buf], 0x3);
                if (++buf == 2) { buf = 0; buf_phase ^= 1; }
            }
        }
    } else {
        // both CTAs: this CTA's 128 rows of the pair's tile, 128 columns to a warp
        const int e = warp - 2, quad = warp & 3, part = e >> 2;
        uint8_t* stg = staging + e * 4096;
        float* bias = biases + e * 128;
        int buf = 0;
        uint32_t buf_phase = 0;
        for (int w = cluster; w < num_tiles; w += nclusters) {
            int tm, tn;
            tiles.coords(w, tm, tn);
            const int row = tm * 2 * BM + (int)rank * BM + quad * 32, col = tn * BN + part * 128;
            stage_bias(a, bias, 128, col, lane);
            if (!mbar_wait(&accf_bar[buf], buf_phase, abort_flag, a.err)) break;
            tc_fence_after();
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {
                float v[64];
                load_sums(tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * BN + part * 128 + g * 64), v);
                if (g == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&acce_bar[buf]), 0));
                }
                if (row < a.M && col + 64 * g < a.N)
                    finish_group(a, &mapY, &mapZ, v, bias + 64 * g, stg, lane, col + 64 * g, row);
            }
            if (++buf == 2) { buf = 0; buf_phase ^= 1; }
        }
        if (lane == 0) bulk_wait_all();
    }
    tc_fence_before();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
    }
}

// ------------------------------------------------------- the slices' sum and epilogue

// P [splits][M][pitch]: four columns to a thread, the slices added in their order
__global__ void __launch_bounds__(256)
    k_fp_join(const float* __restrict__ P, int splits, int64_t stride, int pitch, int M, int N, const FpEpilogue e)
{
    griddep_wait();
    griddep_launch_dependents();
    const int quads = pitch / 4;
    const int64_t n = (int64_t)M * quads;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = i / quads;
        const int c = (int)(i - r * quads) * 4;
        const float* src = P + r * pitch + c;
        float4 s = __ldcs(reinterpret_cast<const float4*>(src));
        for (int q = 1; q < splits; ++q) {
            const float4 v = __ldcs(reinterpret_cast<const float4*>(src + q * stride));
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < N) fp_finish(e, r, c + j, v[j]);
    }
}

// ------------------------------------------------------------------ host

struct FpPlan {
    bool pair;
    int bn, splits, kb_per_split;
};

// A pair's tile takes four times a 128 x 128 tile's work on two SMs; pairs win once their tiles
// occupy at least half of the device's pairs.
static FpPlan fp_plan(int M, int N, int K)
{
    FpPlan p{};
    const int num_kb = (K + 63) / 64;
    p.splits = 1;
    p.kb_per_split = num_kb;
    const int64_t pair_tiles = (int64_t)((M + 255) / 256) * ((N + 255) / 256);
    p.pair = M > 128 && N > 128 && 4 * pair_tiles >= num_sms();
    if (p.pair) return p;
    const int64_t row_tiles = (M + 127) / 128;
    p.bn = row_tiles * ((N + 127) / 128) * 2 <= num_sms() || N <= 64 ? 64 : 128;
    const int64_t tiles = row_tiles * ((N + p.bn - 1) / p.bn);
    // few tiles: slices of at least four K blocks, up to one item per SM
    int64_t splits = num_sms() / tiles;
    if (splits > num_kb / 4) splits = num_kb / 4;
    if (splits > 1) {
        p.kb_per_split = (num_kb + (int)splits - 1) / (int)splits;
        p.splits = (num_kb + p.kb_per_split - 1) / p.kb_per_split;
    }
    return p;
}

static int64_t pad4(int64_t n) { return (n + 3) & ~int64_t(3); }

size_t fp_gemm_ws_bytes(int M, int N, int K)
{
    const FpPlan p = fp_plan(M, N, K);
    return p.splits > 1 ? (size_t)p.splits * M * pad4(N) * sizeof(float) : 0;
}

// 2-D box map (128-byte swizzle) over a row-major tensor of 16-bit or 32-bit elements
static int box_map(CUtensorMap* map, void* p, bool wide, int64_t rows, int64_t cols, int64_t ld, int box_rows)
{
    auto enc = get_encode();
    if (!enc) return set_error(ITO_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    const int size = wide ? 4 : 2;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld * size};
    cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, wide ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, p, dims,
                           strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ITO_OK : set_error(ITO_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

// whether TMA can address the rows: 16-byte aligned base and row stride (a single row's stride is free)
static bool rows_aligned(const void* p, int64_t ld, int size, int64_t rows)
{
    return aligned_to(p, 16) && (ld * size) % 16 == 0 && ld > 0 && (rows == 1 || ld * size < (int64_t(1) << 40));
}

template <typename K>
static cudaError_t allow_smem(K kern, int bytes, bool* done)
{
    if (*done) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    *done = e == cudaSuccess;
    return e;
}

static int max_pairs()
{
    static int n = 0;
    static bool ready = false;
    if (n) return n;
    if (allow_smem(k_fp_gemm_pair, FpPairCfg::SMEM_BYTES, &ready) != cudaSuccess) return 0;
    cudaLaunchConfig_t q = {};
    q.gridDim = dim3(2 * num_sms());
    q.blockDim = dim3(FpPairCfg::THREADS);
    q.dynamicSmemBytes = FpPairCfg::SMEM_BYTES;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    q.attrs = at;
    q.numAttrs = 1;
    int got = 0;
    if (cudaOccupancyMaxActiveClusters(&got, k_fp_gemm_pair, &q) == cudaSuccess && got > 0) n = got;
    return n;
}

template <int BN>
static int launch_single(const CUtensorMap& A, const CUtensorMap& B, const CUtensorMap& Y, const CUtensorMap& Z,
                         const CUtensorMap& S, const FpGemmArgs& a, cudaStream_t s)
{
    static bool ready = false;
    if (allow_smem(k_fp_gemm<BN>, FpCfg<BN>::SMEM_BYTES, &ready) != cudaSuccess)
        return set_error(ITO_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(cudaGetLastError()));
    const int64_t items = (int64_t)((a.M + 127) / 128) * ((a.N + BN - 1) / BN) * a.splits;
    const int grid = items < num_sms() ? (int)items : num_sms();
    launch_pdl(k_fp_gemm<BN>, grid, FpCfg<BN>::THREADS, FpCfg<BN>::SMEM_BYTES, s, A, B, Y, Z, S, a);
    return launch_status("linear product");
}

int fp_gemm(const FpOperand& A, const FpOperand& B, int M, int N, int K, const FpEpilogue& e, void* ws, cudaStream_t s)
{
    const FpPlan p = fp_plan(M, N, K);
    FpGemmArgs a;
    memset(&a, 0, sizeof(a));
    a.e = e;
    a.M = M;
    a.N = N;
    a.K = K;
    a.a_mn = A.mn;
    a.b_mn = B.mn;
    a.group = 16;
    a.splits = p.splits;
    a.kb_per_split = p.kb_per_split;
    a.err = device_error_word();
    if (!a.err) return set_error(ITO_ERR_CUDA, "device error word unavailable");
    const bool wide = e.out_type == ITO_F32;
    a.y_tma = rows_aligned(e.y, e.ldy, wide ? 4 : 2, M);
    a.z_tma = e.z && rows_aligned(e.z, e.ldz, 2, M);
    a.r_vec = e.residual && rows_aligned(e.residual, e.ldr, wide ? 4 : 2, M);
    a.idesc = fp_idesc(p.pair ? 256 : 128, p.pair ? 256 : p.bn, A.mn, B.mn, e.type == ITO_BF16);
    CUtensorMap mA, mB, mY, mZ, mS;
    memset(&mY, 0, sizeof(mY));
    memset(&mZ, 0, sizeof(mZ));
    memset(&mS, 0, sizeof(mS));
    int r = box_map(&mA, const_cast<void*>(A.p), false, A.mn ? K : M, A.mn ? M : K, A.ld, A.mn ? 64 : 128);
    if (!r) r = box_map(&mB, const_cast<void*>(B.p), false, B.mn ? K : N, B.mn ? N : K, B.ld, B.mn ? 64 : p.pair ? 128 : p.bn);
    if (!r && a.y_tma) r = box_map(&mY, e.y, wide, M, N, e.ldy, 32);
    if (!r && a.z_tma) r = box_map(&mZ, e.z, false, M, N, e.ldz, 32);
    if (r) return r;
    if (p.pair) {
        const int tiles = ((M + 255) / 256) * ((N + 255) / 256), most = max_pairs();
        if (!most) return set_error(ITO_ERR_CUDA, "no CTA pair fits on this device");
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (tiles < most ? tiles : most));
        cfg.blockDim = dim3(FpPairCfg::THREADS);
        cfg.dynamicSmemBytes = FpPairCfg::SMEM_BYTES;
        cfg.stream = s;
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 2;
        const cudaError_t ce = cudaLaunchKernelEx(&cfg, k_fp_gemm_pair, mA, mB, mY, mZ, a);
        return ce == cudaSuccess ? ITO_OK : set_error(ITO_ERR_CUDA, "linear product launch: %s", cudaGetErrorString(ce));
    }
    const int64_t pitch = pad4(N);
    if (p.splits > 1) {
        auto enc = get_encode();
        cuuint64_t dims[3] = {(cuuint64_t)pitch, (cuuint64_t)M, (cuuint64_t)p.splits};
        cuuint64_t strides[2] = {(cuuint64_t)pitch * 4, (cuuint64_t)pitch * M * 4};
        cuuint32_t box[3] = {32, 32, 1};
        cuuint32_t estr[3] = {1, 1, 1};
        const CUresult cr = enc(&mS, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, ws, dims, strides, box, estr,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (cr != CUDA_SUCCESS) return set_error(ITO_ERR_CUDA, "cuTensorMapEncodeTiled (partials) failed (%d)", (int)cr);
    }
    r = p.bn == 128 ? launch_single<128>(mA, mB, mY, mZ, mS, a, s) : launch_single<64>(mA, mB, mY, mZ, mS, a, s);
    if (r || p.splits == 1) return r;
    launch_pdl(k_fp_join, launch_grid_blocks((int64_t)M * (pitch / 4), 256), 256, 0, s, static_cast<const float*>(ws),
               p.splits, pitch * M, (int)pitch, M, N, e);
    return launch_status("linear join");
}

}  // namespace ito
