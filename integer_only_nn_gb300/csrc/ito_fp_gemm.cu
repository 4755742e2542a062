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
// feeds twice the work), or narrower ones, for results with enough of them to occupy the device; 128 x 128 and
// 128 x 64 tiles of one CTA, with K cut into slices where there are few tiles, for the rest.
// Slices write their sums in 32 bits to the workspace, and a second kernel adds them in a fixed
// order and does the epilogue. A weight gradient over a long batch is such a product too.
//
// Each kernel is compiled once for each end (FpEnd): the gated layer's two products on one A, the
// parts of a softmax over the columns, the gradient that such a softmax sends back, and gradients in halves.
#include <algorithm>
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
    FpMore x;
    int M, N, K;
    int a_mn, b_mn;
    uint32_t idesc;
    int group, bn;              // row tiles of a raster group; columns of a pair's tile
    int splits, kb_per_split;   // K slices (1: none); slices go to mapS
    int y_tma, z_tma;           // rows of y and z that TMA stores can take
    int r_vec, b_vec;           // rows of the residual, and a bias, that 16-byte loads can take
    int* err;
    // the other ends'
    int y2_tma, z2_tma, b2_vec;
    int cols;                   // result columns of a tile: bn, half of it in the gated layer
    int kb_half;                // K blocks in the first half of B (0: no halves)
    int halves, a_half;         // results from one A
};

// A product's tensor maps and arguments. B2, Y2: a second B, a second result (z2 or y2)
struct FpProblem {
    CUtensorMap A, B, Y, Z, S, B2, Y2;
    FpGemmArgs a;
};

// The producer's and the issuer's warps run their loops whole, so that what they count is uniform
// over the warp, and one elected lane issues: loops of a single lane keep it in ordinary
// registers, and moving it to the uniform ones that copies and products take their operands from
// cost up to a tenth of a product's time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r)::"memory");
    return r != 0;
}

// All lanes wait; whether it came, for all of them alike. Where a wait has run out, in these warps or
// another, the loops end early; then as otherwise the producer stays until its copies have landed
// (ring_landed) and the issuer until the products that free the stages are done, so that no block
// gives its shared or tensor memory back while they are in use. (Of a pair the leader's barrier counts both blocks'
// copies, and the pair leaves together.)
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, err));
}

// Shared-memory descriptors of the K steps of 16 in a stage: 32 bytes on inside the swizzled row
// (K-major), 16 rows of 128 bytes on (MN-major). Addresses count 16 bytes in the descriptor's low
// bits, so a step is one addition; the thread that issues the products has little time to spare.
struct FpSteps {
    uint64_t a0, b0;
    uint32_t a_step, b_step;

    __device__ __forceinline__ FpSteps(const FpGemmArgs& g, uint32_t smem, uint32_t a_bytes)
    {
        a0 = smem_desc_sw128(smem, g.a_mn ? 8192 : 16, 1024);
        b0 = smem_desc_sw128(smem + a_bytes, g.b_mn ? 8192 : 16, 1024);
        a_step = g.a_mn ? 2048 >> 4 : 32 >> 4;
        b_step = g.b_mn ? 2048 >> 4 : 32 >> 4;
    }
    __device__ __forceinline__ uint64_t a(uint32_t at, int k) const { return a0 + (at + k * a_step); }
    __device__ __forceinline__ uint64_t b(uint32_t at, int k) const { return b0 + (at + k * b_step); }
};

// ------------------------------------------------------------------ epilogue
//
// A warp holds 32 rows (its lanes) of 32 columns of sums at a time. Its results go through its
// own buffers of shared memory, 32 rows of 64 bytes (16-byte chunk j of row r at j ^ (r / 2 % 4),
// the 64-byte swizzle), and leave by TMA, which clips them at the tensor's edges, or, where rows
// do not start on 16-byte boundaries, by coalesced plain stores. Two buffers to a warp (four
// measured the same), because the operands' ring needs the room: its loads take about as long
// as four stages' products, and 8192 x 4096 x 4096 takes 160 us with four stages, 144 with five,
// 142 with six (with bias, GELU, z and residual 190, 177, 160).
constexpr int kFpBox = 2048, kFpBoxes = 2;

struct FpStage {
    uint8_t* p;
    int lane, turn;

    // the next buffer. Every box is one group of bulk stores (an empty one, where it went by plain
    // stores), so the buffer's last box is kFpBoxes groups back.
    __device__ __forceinline__ uint8_t* begin()
    {
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kFpBoxes - 1) : "memory");
        __syncwarp();
        uint8_t* r = p + turn * kFpBox;
        turn = (turn + 1) % kFpBoxes;
        return r;
    }
};

__device__ __forceinline__ void box_end_tma(const CUtensorMap* map, const uint8_t* stg, int lane, int col, int row)
{
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(map, stg, col, row);
        bulk_commit();
    }
}

// the 4-byte word `w` of a box's row r
__device__ __forceinline__ uint32_t box_word(const uint8_t* stg, int r, int w)
{
    return *reinterpret_cast<const uint32_t*>(stg + r * 64 + (((w >> 2) ^ (r >> 1 & 3)) << 4) + (w & 3) * 4);
}

// 32 columns as 16-bit floats: one box
__device__ __forceinline__ void store16(const float (&v)[32], int type, const CUtensorMap* map, bool tma, void* out,
                                        int64_t ld, FpStage& st, int col, int row, int M, int N)
{
    uint8_t* stg = st.begin();
    const int lane = st.lane;
    const uint32_t at = smem_u32(stg) + lane * 64;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        st_shared_v4(at + ((j ^ (lane >> 1 & 3)) << 4), (int)pack16(type, v[8 * j], v[8 * j + 1]),
                     (int)pack16(type, v[8 * j + 2], v[8 * j + 3]), (int)pack16(type, v[8 * j + 4], v[8 * j + 5]),
                     (int)pack16(type, v[8 * j + 6], v[8 * j + 7]));
    if (tma) {
        box_end_tma(map, stg, lane, col, row);
        return;
    }
    __syncwarp();
    // half a warp to a row, a word of two columns to a lane; in a row that starts on an odd element the
    // words are shifted by one, and its first element is stored alone
    const int w = lane & 15, cols = min(32, N - col);
    uint16_t* dst = static_cast<uint16_t*>(out) + (int64_t)(row + (lane >> 4)) * ld + col;
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += 16) {
        uint32_t x[8], next[8];                  // eight rows' words before their stores
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = box_word(stg, r0 + 2 * k + (lane >> 4), w);
#pragma unroll
        for (int k = 0; k < 8; ++k) next[k] = __shfl_down_sync(0xffffffffu, x[k], 1, 16);
#pragma unroll
        for (int k = 0; k < 8; ++k, dst += 2 * ld) {
            const bool in = row + r0 + 2 * k + (lane >> 4) < M;
            const bool odd = reinterpret_cast<uintptr_t>(dst) & 2;
            const int at = 2 * w + odd;          // columns at and at + 1 of the box
            const uint32_t y = odd ? __funnelshift_r(x[k], next[k], 16) : x[k];
            if (in && at + 1 < cols) *reinterpret_cast<uint32_t*>(dst + at) = y;
            if (in && at + 1 == cols) dst[at] = (uint16_t)y;
            if (in && odd && w == 0) dst[0] = (uint16_t)x[k];
        }
    }
    __syncwarp();
    if (lane == 0) bulk_commit();
}

// 16 of the columns (half h) as 32-bit floats, staged
__device__ __forceinline__ uint8_t* stage32(const float (&v)[32], int h, FpStage& st)
{
    uint8_t* stg = st.begin();
    const int lane = st.lane;
    const uint32_t at = smem_u32(stg) + lane * 64;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = 16 * h + 4 * j;
        st_shared_v4(at + ((j ^ (lane >> 1 & 3)) << 4), __float_as_int(v[i]), __float_as_int(v[i + 1]),
                     __float_as_int(v[i + 2]), __float_as_int(v[i + 3]));
    }
    return stg;
}

// 32 columns as 32-bit floats: two boxes
__device__ __forceinline__ void store32(const float (&v)[32], const CUtensorMap* map, bool tma, void* out, int64_t ld,
                                        FpStage& st, int col, int row, int M, int N)
{
    const int lane = st.lane;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = col + 16 * h;
        if (c >= N) break;
        uint8_t* stg = stage32(v, h, st);
        if (tma) {
            box_end_tma(map, stg, lane, c, row);
            continue;
        }
        __syncwarp();
        const int w = lane & 15;
        for (int r = lane >> 4; r < 32 && row + r < M; r += 2)
            if (c + w < N) static_cast<uint32_t*>(out)[(row + r) * ld + c + w] = box_word(stg, r, w);
        __syncwarp();
        if (lane == 0) bulk_commit();
    }
}

template <int ACT>
__device__ __forceinline__ void activate(float (&v)[32])
{
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const float2 y = act_value<ACT>(make_float2(v[i], v[i + 1]));
        v[i] = y.x;
        v[i + 1] = y.y;
    }
}

__device__ __forceinline__ void activate(int act, float (&v)[32])
{
    switch (act) {
    case ITO_ACT_RELU: activate<ITO_ACT_RELU>(v); break;
    case ITO_ACT_GELU: activate<ITO_ACT_GELU>(v); break;
    case ITO_ACT_GELU_TANH: activate<ITO_ACT_GELU_TANH>(v); break;
    case ITO_ACT_SILU: activate<ITO_ACT_SILU>(v); break;
    default: break;
    }
}

// this lane's row of a 16-bit residual, 32 columns (0 beyond the edges); asked for before the
// sums are there
__device__ __forceinline__ void load_residual16(const FpGemmArgs& a, int col, int row, uint32_t (&w)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 0u;
    if (row >= a.M || col >= a.N) return;
    const uint16_t* r = static_cast<const uint16_t*>(a.e.residual) + row * a.e.ldr + col;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (a.r_vec && col + 8 * j + 8 <= a.N) {
            const uint4 q = *reinterpret_cast<const uint4*>(r + 8 * j);
            w[4 * j] = q.x;
            w[4 * j + 1] = q.y;
            w[4 * j + 2] = q.z;
            w[4 * j + 3] = q.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + 8 * j + i < a.N) w[4 * j + (i >> 1)] |= (uint32_t)r[8 * j + i] << (16 * (i & 1));
        }
    }
}

// the columns' biases, the same for every lane; vec: 16-byte loads can take them
__device__ __forceinline__ void add_bias(const void* bias, int type, int vec, int N, float (&v)[32], int col)
{
    if (vec && col + 32 <= N && type != ITO_F32) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(bias) + col);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 q = __ldg(p + j);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack16(type, w[i]);
                v[8 * j + 2 * i] += f.x;
                v[8 * j + 2 * i + 1] += f.y;
            }
        }
    } else if (vec && col + 32 <= N) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(bias) + col);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 q = __ldg(p + j);
            v[4 * j] += q.x;
            v[4 * j + 1] += q.y;
            v[4 * j + 2] += q.z;
            v[4 * j + 3] += q.w;
        }
    } else {
        const int c = col + (threadIdx.x & 31);
        const float mine = c < N ? load_typed(bias, type, c) : 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xffffffffu, mine, i);
    }
}

// `left` elements of a row of 32-bit floats added (32 at most)
__device__ __forceinline__ void add_row32(const float* r, int vec, int left, float (&v)[32])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (vec && 4 * j + 4 <= left) {
            const float4 q = *reinterpret_cast<const float4*>(r + 4 * j);
            v[4 * j] += q.x;
            v[4 * j + 1] += q.y;
            v[4 * j + 2] += q.z;
            v[4 * j + 3] += q.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * j + i < left) v[4 * j + i] += r[4 * j + i];
        }
    }
}

__device__ __forceinline__ void finish_group(const FpGemmArgs& a, const CUtensorMap* mapY, const CUtensorMap* mapZ,
                                             float (&v)[32], const uint32_t (&res)[16], FpStage& st, int col, int row)
{
    const FpEpilogue& e = a.e;
    const int lane = st.lane;
    if (e.bias) add_bias(e.bias, e.bias_type, a.b_vec, a.N, v, col);
    if (e.z) store16(v, e.type, mapZ, a.z_tma, e.z, e.ldz, st, col, row, a.M, a.N);
    activate(e.act, v);
    if (e.out_type != ITO_F32) {
        if (e.residual) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 f = unpack16(e.out_type, res[i]);
                v[2 * i] += f.x;
                v[2 * i + 1] += f.y;
            }
        }
        store16(v, e.out_type, mapY, a.y_tma, e.y, e.ldy, st, col, row, a.M, a.N);
        return;
    }
    if (e.residual && row + lane < a.M)
        add_row32(static_cast<const float*>(e.residual) + (row + lane) * e.ldr + col, a.r_vec, a.N - col, v);
    store32(v, mapY, a.y_tma, e.y, e.ldy, st, col, row, a.M, a.N);
}

// zg and zu of a gated layer: both biases, both saved, h = act(zg) zu
__device__ __forceinline__ void finish_gated(const FpProblem& p, float (&g)[32], float (&u)[32], FpStage& st, int col,
                                             int row)
{
    const FpGemmArgs& a = p.a;
    const FpEpilogue& e = a.e;
    if (e.bias) add_bias(e.bias, e.bias_type, a.b_vec, a.N, g, col);
    if (a.x.bias2) add_bias(a.x.bias2, e.bias_type, a.b2_vec, a.N, u, col);
    if (e.z) {
        store16(g, e.type, &p.Z, a.z_tma, e.z, e.ldz, st, col, row, a.M, a.N);
        store16(u, e.type, &p.Y2, a.z2_tma, a.x.z2, a.x.ldz2, st, col, row, a.M, a.N);
    }
    activate(e.act, g);
#pragma unroll
    for (int i = 0; i < 32; ++i) g[i] *= u[i];
    store16(g, e.type, &p.Y, a.y_tma, e.y, e.ldy, st, col, row, a.M, a.N);
}

// a gradient's sums: *alpha sum + acc
__device__ __forceinline__ void finish_grad(const FpProblem& p, int half, float (&v)[32], FpStage& st, int col, int row)
{
    const FpGemmArgs& a = p.a;
    const FpEpilogue& e = a.e;
    if (a.x.alpha) {
        const float alpha = __ldg(a.x.alpha);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= alpha;
    }
    if (a.x.acc && row + st.lane < a.M) add_row32(a.x.acc + (row + st.lane) * a.x.ldacc + col, a.r_vec, a.N - col, v);
    const CUtensorMap* map = half ? &p.Y2 : &p.Y;
    const bool tma = half ? a.y2_tma : a.y_tma;
    void* y = half ? a.x.y2 : e.y;
    const int64_t ld = half ? a.x.ldy2 : e.ldy;
    if (e.out_type == ITO_F32) store32(v, map, tma, y, ld, st, col, row, a.M, a.N);
    else store16(v, e.out_type, map, tma, y, ld, st, col, row, a.M, a.N);
}

// a warp's wait: one lane asks
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err)
{
    bool ok = true;
    if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort_flag, err);
    return __shfl_sync(0xffffffffu, ok, 0);
}

__device__ __forceinline__ void load_sums(uint32_t taddr, float (&v)[32])
{
    uint32_t r[32];
    tmem_ld32(taddr, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void load_sums(uint32_t first, uint32_t second, float (&v)[32], float (&u)[32])
{
    uint32_t r[32], q[32];
    tmem_ld32(first, r);
    tmem_ld32(second, q);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i] = __uint_as_float(r[i]);
        u[i] = __uint_as_float(q[i]);
    }
}

// ------------------------------------------------------- a softmax's parts and its gradient

// One lane's row of a tile: its class, and the running largest sum m and s = sum of exp(sum - m).
// A sum of -inf adds 0; a NaN or an infinity makes s a NaN.
struct LossRow {
    int target;
    float m, s;

    // 32 columns from col on, of which `left` exist; -> the target's sum to *hit, where it is among them
    __device__ __forceinline__ void add(float (&v)[32], int col, int left, float* hit)
    {
        if (left < 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i >= left) v[i] = -INFINITY;
        }
        const int at = target - col;
        if (at >= 0 && at < 32) {
            float x = v[0];
#pragma unroll
            for (int i = 1; i < 32; ++i)
                if (i == at) x = v[i];
            *hit = x;
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < 32; ++i) top = fmaxf(top, v[i]);
        const float ref = top == -INFINITY ? 0.0f : top;
        s *= exp2_approx((m - ref) * kFpLog2e);
        float t[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            t[0] += exp2_approx((v[i] - ref) * kFpLog2e);
            t[1] += exp2_approx((v[i + 1] - ref) * kFpLog2e);
        }
        s += t[0] + t[1];
        m = top;
    }
};

// The tensor cores cut off what a sum's 24 bits cannot hold, at each step of 16 k: a chain of 256 steps
// leaves logits short by 2^-17 of their size, and lse by 1.5e-6 of its own (4096 x 4096 -> 32768). So a
// logit's sums are taken out of tensor memory every kLogitChunk K blocks and added up in registers,
// rounded: one accumulator is added while the other fills. The gradient's logits (DLogits) are summed as the Loss's
// were, bit for bit: exp(l - lse) - 1 of a row whose target has nearly all of the probability is a difference
// of neighbours, of which a logit short by 2^-17 leaves nothing right from p = 0.9999 on.
constexpr int kLogitChunk = 16;
template <FpEnd END>
constexpr bool kLogits = END == FpEnd::Loss || END == FpEnd::DLogits;

// Whether a tile with K blocks lo .. hi - 1 is drained in chunks. A DLogits tile of one chunk is not: the sums are the
// same, and each 32 columns leave as soon as they are read (512 x 512 x 8192, both gradients, us: 26.4, in chunks 27.8).
template <FpEnd END>
__device__ __forceinline__ bool in_chunks(int lo, int hi)
{
    return END == FpEnd::Loss || (END == FpEnd::DLogits && hi - lo > kLogitChunk);
}

// K blocks from one drain of the accumulator to the next
template <FpEnd END>
__device__ __forceinline__ int chunk_end(int kb, int hi)
{
    return kLogits<END> ? min(hi, kb + kLogitChunk) : hi;
}

// The epilogue of a tile of logits: as drain_tile, over all `chunks` of the tile's K range. ready() waits for a
// chunk's sums and gives their place in tensor memory, done() tells that they are read.
template <FpEnd END, int MAX_COLS, typename Ready, typename Done>
__device__ __forceinline__ void drain_logits(const FpProblem& p, int slice, FpStage& st, int first, int columns, int col0,
                                             int row, int chunks, Ready ready, Done done, bool& ok)
{
    constexpr int GROUPS = MAX_COLS / 64;            // (two warps to a row quarter)
    const FpGemmArgs& a = p.a;
    const int lane = st.lane;
    LossRow loss;
    SlopeRow slope;
    if (END == FpEnd::Loss) loss = LossRow{row + lane < a.M ? a.x.targets[row + lane] : -1, -INFINITY, 0.0f};
    else slope.load(a.x, a.M, row + lane, first == 0 && col0 == 0 && a.x.first == 0, a.err);
    float sum[GROUPS][32];
#pragma unroll
    for (int g = 0; g < GROUPS; ++g)
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[g][i] = 0.0f;
#pragma unroll 1
    for (int q = 0; q < chunks; ++q) {
        uint32_t taddr;
        if (!ready(taddr)) {
            ok = false;
            return;
        }
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const int c = (first + 2 * g) * 32;
            if (c < columns) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {        // (16 at a time: the sums leave few registers)
                    uint32_t v[16];
                    tmem_ld16(taddr + c + 16 * h, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[g][16 * h + i] += __uint_as_float(v[i]);
                }
            }
        }
        tc_fence_before();
        __syncwarp();
        done();
    }
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        const int c = (first + 2 * g) * 32;
        if (c >= columns || row >= a.M || col0 + c >= a.N) continue;
        if (slice < 0 && END == FpEnd::Loss) {
            loss.add(sum[g], col0 + c, a.N - col0 - c, a.x.hit + row + lane);
            continue;
        }
        if (slice < 0) {
            slope.apply(sum[g], col0 + c);
            store16(sum[g], a.e.type, &p.Y, true, a.e.y, a.e.ldy, st, col0 + c, row, a.M, a.N);
            continue;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (col0 + c + 16 * h >= a.N) break;
            uint8_t* stg = stage32(sum[g], h, st);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_3d(&p.S, stg, col0 + c + 16 * h, row, slice);
                bulk_commit();
            }
        }
    }
    if (END == FpEnd::Loss && slice < 0 && row + lane < a.M)
        a.x.part[(int64_t)(col0 / columns * 2 + first) * a.M + row + lane] = make_float2(loss.m, loss.s);
}

// The epilogue of the groups of 32 columns first, first + step, .. below `columns` of a tile at
// (row, col0), sums at `taddr`; `done` tells the issuing warp that the accumulator is drained. A
// slice of K (slice >= 0) leaves its sums as they are, in the workspace. `half`: of a result in halves.
template <FpEnd END, typename Wait, typename Done>
__device__ __forceinline__ void drain_tile(const FpProblem& p, int slice, int half, FpStage& st, int first, int step,
                                           int columns, int col0, int row, uint32_t taddr, Wait wait, Done done,
                                           bool& ok)
{
    const FpGemmArgs& a = p.a;
    // a 16-bit residual comes while the sums are still being made
    const bool res16 = END == FpEnd::Linear && slice < 0 && a.e.residual && a.e.out_type != ITO_F32;
    uint32_t res[16];
    if (res16) load_residual16(a, col0 + first * 32, row + st.lane, res);
    SlopeRow slope;
    if (END == FpEnd::DLogits) slope.load(a.x, a.M, row + st.lane, first == 0 && col0 == 0 && a.x.first == 0, a.err);
    if (!wait()) {
        ok = false;
        return;
    }
    tc_fence_after();
#pragma unroll 1
    for (int c = first * 32; c < columns; c += step * 32) {
        float v[32], u[32];
        if (END == FpEnd::Gated) load_sums(taddr + c, taddr + columns + c, v, u);
        else load_sums(taddr + c, v);
        if (c + step * 32 >= columns) {
            tc_fence_before();
            __syncwarp();
            done();
        }
        if (row >= a.M || col0 + c >= a.N) continue;
        if (slice >= 0) {
            constexpr int PLANES = END == FpEnd::Gated ? 2 : 1;
            const int plane = END == FpEnd::Gated ? 2 * slice : END == FpEnd::Grad ? a.halves * slice + half : slice;
#pragma unroll
            for (int h = 0; h < 2 * PLANES; ++h) {
                if (col0 + c + 16 * (h & 1) >= a.N) continue;
                uint8_t* stg = stage32(h < 2 ? v : u, h & 1, st);
                fence_proxy_async_smem();
                __syncwarp();
                if (st.lane == 0) {
                    tma_store_3d(&p.S, stg, col0 + c + 16 * (h & 1), row, plane + (h >> 1));
                    bulk_commit();
                }
            }
            continue;
        }
        if (END == FpEnd::Linear) {
            if (res16 && c > first * 32) load_residual16(a, col0 + c, row + st.lane, res);
            finish_group(a, &p.Y, &p.Z, v, res, st, col0 + c, row);
        } else if (END == FpEnd::Gated) {
            finish_gated(p, v, u, st, col0 + c, row);
        } else if (END == FpEnd::DLogits) {
            slope.apply(v, col0 + c);
            store16(v, a.e.type, &p.Y, true, a.e.y, a.e.ldy, st, col0 + c, row, a.M, a.N);
        } else {
            finish_grad(p, half, v, st, col0 + c, row);
        }
    }
}

// Tells the pair's leader that this warp has read its part of an accumulator. What the arrival orders are reads of
// tensor memory, complete since tcgen05.wait::ld; a release at the cluster's scope would wait for the warp's
// stores to global memory as well: 2000 to 3000 cycles a tile, which bounds products of a short K.
__device__ __forceinline__ void mbar_arrive_drained(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// ----------------------------------------------------------------- one CTA

template <int BN>
struct FpCfg {
    static constexpr int BM = 128, BK = 64;
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int EPI_WARPS = 8;                  // two to a quarter of the rows
    static constexpr int THREADS = 64 + EPI_WARPS * 32;
    static constexpr int TMEM_COLS = 2 * BN;
    static constexpr int STAGES = BN == 128 ? 6 : 8;
    static constexpr int STAGING_BYTES = EPI_WARPS * kFpBoxes * kFpBox;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + STAGING_BYTES + 1024 + 256;
};

template <int BN, FpEnd END>
__global__ void __launch_bounds__(FpCfg<BN>::THREADS, 1) k_fp_gemm(const __grid_constant__ FpProblem p)
{
    using Cfg = FpCfg<BN>;
    constexpr int COLS = END == FpEnd::Gated ? BN / 2 : BN;      // result columns of a tile
    const FpGemmArgs& a = p.a;
    constexpr int BM = Cfg::BM, BK = Cfg::BK, STAGES = Cfg::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* staging = smem + STAGES * Cfg::STAGE_BYTES;
    uint64_t* full_bar = reinterpret_cast<uint64_t*>(staging + Cfg::STAGING_BYTES);
    uint64_t* empty_bar = full_bar + STAGES;
    uint64_t* accf_bar = empty_bar + STAGES;
    uint64_t* acce_bar = accf_bar + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce_bar + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int num_m = (a.M + BM - 1) / BM;                       // row tiles of a result
    const FpTiles tiles{END == FpEnd::Grad ? num_m * a.halves : num_m, (a.N + COLS - 1) / COLS, a.group};
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
        prefetch_tensormap(&p.A);
        prefetch_tensormap(&p.B);
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
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int w = blockIdx.x; ok && w < num_items; w += gridDim.x) {
            int tm, tn;
            tiles.coords(w / a.splits, tm, tn);
            const int lo = (w % a.splits) * a.kb_per_split, hi = min(num_kb, lo + a.kb_per_split);
            int rowA = tm * BM;
            if (END == FpEnd::Grad && tm >= num_m) rowA = a.a_half + (tm - num_m) * BM;
            for (int kb = lo; kb < hi; ++kb) {
                if (!ring_wait(&empty_bar[stage], phase ^ 1, abort_flag, a.err)) { ok = false; break; }
                if (elect_one()) {
                    mbar_arrive_expect_tx(&full_bar[stage], Cfg::STAGE_BYTES);
                    uint8_t* sA = smem + stage * Cfg::STAGE_BYTES;
                    uint8_t* sB = sA + Cfg::A_BYTES;
                    if (!a.a_mn) {
                        tma_load_2d(&p.A, &full_bar[stage], sA, kb * BK, rowA);
                    } else {
                        tma_load_2d(&p.A, &full_bar[stage], sA, rowA, kb * BK);
                        tma_load_2d(&p.A, &full_bar[stage], sA + 8192, rowA + 64, kb * BK);
                    }
                    if (END == FpEnd::Gated) {           // (both K-major; boxes of COLS rows)
                        tma_load_2d(&p.B, &full_bar[stage], sB, kb * BK, tn * COLS);
                        tma_load_2d(&p.B2, &full_bar[stage], sB + Cfg::B_BYTES / 2, kb * BK, tn * COLS);
                    } else if (!a.b_mn) {
                        tma_load_2d(&p.B, &full_bar[stage], sB, kb * BK, tn * BN);
                    } else {
                        const bool second = END == FpEnd::Grad && a.kb_half && kb >= a.kb_half;
                        const CUtensorMap* map = second ? &p.B2 : &p.B;
                        const int k = second ? kb - a.kb_half : kb;
#pragma unroll
                        for (int j = 0; j < BN / 64; ++j)
                            tma_load_2d(map, &full_bar[stage], sB + j * 8192, tn * BN + j * 64, k * BK);
                    }
                }
                __syncwarp();
                if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
        }
        if (lane == 0) ring_landed(full_bar, STAGES, RingPlace{stage, phase}.lap_before(), STAGES);
    } else if (warp == 1) {
        int stage = 0, buf = 0;
        uint32_t phase = 0, buf_phase = 0;
        bool ok = true;
        const FpSteps step(a, smem_u32(smem), Cfg::A_BYTES);
        const uint32_t idesc = a.idesc;
        for (int w = blockIdx.x; ok && w < num_items; w += gridDim.x) {
            const int first = (w % a.splits) * a.kb_per_split, end = min(num_kb, first + a.kb_per_split);
            for (int lo = first, hi; ok && lo < end; lo = hi) {
                hi = chunk_end<END>(lo, end);
                if (!ring_wait(&acce_bar[buf], buf_phase ^ 1, abort_flag, a.err)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(buf * BN);
                for (int kb = lo; kb < hi; ++kb) {
                    if (!ring_wait(&full_bar[stage], phase, abort_flag, a.err)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t at = (uint32_t)stage * (Cfg::STAGE_BYTES >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < BK / 16; ++k)
                            tc_mma_bf16(d, step.a(at, k), step.b(at, k), idesc, (kb > lo || k > 0) ? 1u : 0u);
                        tc_commit(&empty_bar[stage]);
                        if (kb + 1 == hi) tc_commit(&accf_bar[buf]);
                    }
                    __syncwarp();
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
                if (++buf == 2) { buf = 0; buf_phase ^= 1; }
            }
        }
        if (lane == 0) ring_landed(empty_bar, STAGES, RingPlace{stage, phase}.lap_before(), STAGES);
    } else {
        const int e = warp - 2, quad = warp & 3, part = e >> 2;
        FpStage st{staging + e * kFpBoxes * kFpBox, lane, 0};
        int buf = 0;
        uint32_t buf_phase = 0;
        bool ok = true;
        for (int w = blockIdx.x; ok && w < num_items; w += gridDim.x) {
            int tm, tn;
            tiles.coords(w / a.splits, tm, tn);
            const int half = END == FpEnd::Grad && tm >= num_m;
            if constexpr (kLogits<END>) {
                const int lo = (w % a.splits) * a.kb_per_split, hi = min(num_kb, lo + a.kb_per_split);
                if (in_chunks<END>(lo, hi)) {
                    drain_logits<END, BN>(
                        p, a.splits > 1 ? w % a.splits : -1, st, part, COLS, tn * COLS, tm * BM + quad * 32,
                        (hi - lo + kLogitChunk - 1) / kLogitChunk,
                        [&](uint32_t& taddr) {
                            taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * BN);
                            return warp_wait(&accf_bar[buf], buf_phase, abort_flag, a.err);
                        },
                        [&] {
                            if (lane == 0) mbar_arrive(&acce_bar[buf]);
                            if (++buf == 2) { buf = 0; buf_phase ^= 1; }
                        },
                        ok);
                    continue;
                }
            }
            drain_tile<END>(
                p, a.splits > 1 ? w % a.splits : -1, half, st, part, 2, COLS, tn * COLS,
                (half ? tm - num_m : tm) * BM + quad * 32,
                tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * BN),
                [&] { return warp_wait(&accf_bar[buf], buf_phase, abort_flag, a.err); },
                [&] { if (lane == 0) mbar_arrive(&acce_bar[buf]); }, ok);
            if (++buf == 2) { buf = 0; buf_phase ^= 1; }
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

// A tile is 256 rows by a.bn columns, 256 or fewer (a multiple of 32), so that the tiles of a
// result come out near whole waves: 2048 x 4096 is 128 tiles of 256 columns, two waves of the
// 76 pairs of which the second is two thirds full, or 152 tiles of 224 columns, two full ones.
struct FpPairCfg {
    static constexpr int BM = 128, MAX_BN = 256, BK = 64;
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = (MAX_BN / 2) * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = 6;
    static constexpr int EPI_WARPS = 8;
    static constexpr int THREADS = 64 + EPI_WARPS * 32;
    static constexpr int TMEM_COLS = 512;
    static constexpr int STAGING_BYTES = EPI_WARPS * kFpBoxes * kFpBox;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + STAGING_BYTES + 1024 + 256;
};

// One product, or two in one launch (the backward pass's), so that the second's items (tiles, or
// their K slices) fill the first's last wave. The items of problem 0, whose K range is the longer
// one, go round the pairs; of its last round `rest` pairs have one, and the others meanwhile take
// `gap` items each of problem 1, whose remaining items go round all pairs. At 2048 x 4096 x 4096 the two products
// are 2 + 4 waves one by one, 7/8 of that together. A launch of one product has a kernel of its
// own: with the second one's branches 8192 x 4096 x 4096 takes 145 us instead of 142, and 171 instead of
// 160 with bias, GELU, z and residual.
template <int PROBLEMS>
struct FpPairWork {
    FpProblem p[PROBLEMS];
    int items[2];
    int rest, gap;

    // item k of pair c of C
    __device__ __forceinline__ bool item(int k, int c, int C, int& problem, int& i) const
    {
        if (PROBLEMS == 1) {
            problem = 0;
            i = c + k * C;
            return i < items[0];
        }
        const int n = c < items[0] ? (items[0] - 1 - c) / C + 1 : 0;
        problem = 0;
        i = c + k * C;
        if (k < n) return true;
        k -= n;
        problem = 1;
        if (gap && c >= rest) {
            i = k * (C - rest) + c - rest;
            if (k < gap) return i < items[1];
            k -= gap;
        }
        i = gap * (C - rest) + k * C + c;
        return i < items[1];
    }
};

template <int PROBLEMS, FpEnd END>
__global__ void __launch_bounds__(FpPairCfg::THREADS, 1)
    k_fp_gemm_pair(const __grid_constant__ FpPairWork<PROBLEMS> work)
{
    constexpr int LAST = PROBLEMS - 1;
    using Cfg = FpPairCfg;
    constexpr int BM = Cfg::BM, BK = Cfg::BK, STAGES = Cfg::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* staging = smem + STAGES * Cfg::STAGE_BYTES;
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
    int* const err = work.p[0].a.err;

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
#pragma unroll
        for (int i = 0; i < PROBLEMS; ++i) {
            prefetch_tensormap(&work.p[i].A);
            prefetch_tensormap(&work.p[i].B);
        }
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

    // an item's place in its result (and which, of two halves), and its K blocks
    auto place = [&](const FpGemmArgs& a, int item, int& row, int& col, int& half) {
        const int cols = END == FpEnd::Gated ? a.cols : a.bn, num_m = (a.M + 2 * BM - 1) / (2 * BM);
        const FpTiles tiles{END == FpEnd::Grad ? num_m * a.halves : num_m, (a.N + cols - 1) / cols, a.group};
        int tm, tn;
        tiles.coords(item / a.splits, tm, tn);
        half = END == FpEnd::Grad && tm >= num_m;
        if (half) tm -= num_m;
        row = tm * 2 * BM + (int)rank * BM;
        col = tn * cols;
    };
    auto k_range = [&](const FpGemmArgs& a, int item, int& lo, int& hi) {
        lo = item % a.splits * a.kb_per_split;
        hi = min((a.K + BK - 1) / BK, lo + a.kb_per_split);
    };
    int problem, item;
    if (warp == 0) {
        // both CTAs load; every load completes on the leader's barrier. (An MN-major B comes in
        // whole boxes of 64 columns, some beyond a narrow tile's half.)
        {
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            const uint32_t bar0 = mapa_shared(smem_u32(&full_bar[0]), 0);
            auto load = [&](const FpProblem& p) {
                const FpGemmArgs& a = p.a;
                const bool a_mn = a.a_mn, b_mn = a.b_mn;
                const uint32_t stage_bytes = 2 * (Cfg::A_BYTES + (b_mn ? Cfg::B_BYTES : (a.bn / 2) * BK * 2));
                int rowA, rowB, half, lo, hi;
                place(a, item, rowA, rowB, half);
                k_range(a, item, lo, hi);
                if (half) rowA += a.a_half;
                // of the gated layer's two products each CTA stages its own one's B
                const CUtensorMap* mapB = END == FpEnd::Gated && !leader ? &p.B2 : &p.B;
                if (END != FpEnd::Gated) rowB += (int)rank * (a.bn / 2);
                for (int kb = lo; kb < hi; ++kb) {
                    if (!ring_wait(&empty_bar[stage], phase ^ 1, abort_flag, err)) { ok = false; break; }
                    if (elect_one()) {
                        if (leader) mbar_arrive_expect_tx(&full_bar[stage], stage_bytes);
                        const uint32_t fb = bar0 + stage * 8;
                        uint8_t* sA = smem + stage * Cfg::STAGE_BYTES;
                        uint8_t* sB = sA + Cfg::A_BYTES;
                        if (!a_mn) {
                            tma_load_2d_pair(&p.A, fb, sA, kb * BK, rowA);
                        } else {
                            tma_load_2d_pair(&p.A, fb, sA, rowA, kb * BK);
                            tma_load_2d_pair(&p.A, fb, sA + 8192, rowA + 64, kb * BK);
                        }
                        if (!b_mn) {
                            tma_load_2d_pair(mapB, fb, sB, kb * BK, rowB);
                        } else {
                            const bool second = END == FpEnd::Grad && a.kb_half && kb >= a.kb_half;
                            const CUtensorMap* map = second ? &p.B2 : mapB;
                            const int k = second ? kb - a.kb_half : kb;
                            tma_load_2d_pair(map, fb, sB, rowB, k * BK);
                            tma_load_2d_pair(map, fb, sB + 8192, rowB + 64, k * BK);
                        }
                    }
                    __syncwarp();
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
            };
            for (int k = 0; ok && work.item(k, cluster, nclusters, problem, item); ++k) {
                if (PROBLEMS == 1 || problem == 0) load(work.p[0]);
                else load(work.p[LAST]);
            }
            if (leader && lane == 0) ring_landed(full_bar, STAGES, RingPlace{stage, phase}.lap_before(), STAGES);
        }
    } else if (warp == 1) {
        if (leader) {
            int stage = 0, buf = 0;
            uint32_t phase = 0, buf_phase = 0;
            bool ok = true;
            for (int k = 0; ok && work.item(k, cluster, nclusters, problem, item); ++k) {
                const FpGemmArgs& a = PROBLEMS == 1 || problem == 0 ? work.p[0].a : work.p[LAST].a;
                const FpSteps step(a, smem_u32(smem), Cfg::A_BYTES);
                const uint32_t idesc = a.idesc;
                int first, end;
                k_range(a, item, first, end);
                for (int lo = first, hi; ok && lo < end; lo = hi) {
                    hi = chunk_end<END>(lo, end);
                    if (!ring_wait(&acce_bar[buf], buf_phase ^ 1, abort_flag, err)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t d = tmem_base + (uint32_t)(buf * Cfg::MAX_BN);
                    for (int kb = lo; kb < hi; ++kb) {
                        if (!ring_wait(&full_bar[stage], phase, abort_flag, err)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t at = (uint32_t)stage * (Cfg::STAGE_BYTES >> 4);
                        if (elect_one()) {
#pragma unroll
                            for (int q = 0; q < BK / 16; ++q)
                                tc_mma_bf16_pair(d, step.a(at, q), step.b(at, q), idesc, (kb > lo || q > 0) ? 1u : 0u);
                            tc_commit_pair_mc(&empty_bar[stage], 0x3);
                            if (kb + 1 == hi) tc_commit_pair_mc(&accf_bar[buf], 0x3);
                        }
                        __syncwarp();
                        if (++stage == STAGES) { stage = 0; phase ^= 1; }
                    }
                    if (++buf == 2) { buf = 0; buf_phase ^= 1; }
                }
            }
            if (lane == 0) ring_landed(empty_bar, STAGES, RingPlace{stage, phase}.lap_before(), STAGES);
        }
    } else {
        // both CTAs: this CTA's 128 rows of the pair's tile, two warps to 32 of them
        const int e = warp - 2, quad = warp & 3, part = e >> 2;
        FpStage st{staging + e * kFpBoxes * kFpBox, lane, 0};
        int buf = 0;
        uint32_t buf_phase = 0;
        bool ok = true;
        for (int k = 0; ok && work.item(k, cluster, nclusters, problem, item); ++k) {
            const FpProblem& p = PROBLEMS == 1 || problem == 0 ? work.p[0] : work.p[LAST];
            int row, col, half;
            place(p.a, item, row, col, half);
            if constexpr (kLogits<END>) {
                int lo, hi;
                k_range(p.a, item, lo, hi);
                if (in_chunks<END>(lo, hi)) {
                    drain_logits<END, Cfg::MAX_BN>(
                        p, p.a.splits > 1 ? item % p.a.splits : -1, st, part, p.a.bn, col, row + quad * 32,
                        (hi - lo + kLogitChunk - 1) / kLogitChunk,
                        [&](uint32_t& taddr) {
                            taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * Cfg::MAX_BN);
                            return warp_wait(&accf_bar[buf], buf_phase, abort_flag, err);
                        },
                        [&] {
                            if (lane == 0) mbar_arrive_drained(mapa_shared(smem_u32(&acce_bar[buf]), 0));
                            if (++buf == 2) { buf = 0; buf_phase ^= 1; }
                        },
                        ok);
                    continue;
                }
            }
            drain_tile<END>(
                p, p.a.splits > 1 ? item % p.a.splits : -1, half, st, part, Cfg::EPI_WARPS / 4,
                END == FpEnd::Gated ? p.a.cols : p.a.bn, col, row + quad * 32,
                tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * Cfg::MAX_BN),
                [&] { return warp_wait(&accf_bar[buf], buf_phase, abort_flag, err); },
                [&] { if (lane == 0) mbar_arrive_drained(mapa_shared(smem_u32(&acce_bar[buf]), 0)); }, ok);
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

// P [splits][M][pitch], or [splits][2][M][pitch] with a second sum of each element or for each half:
// four columns to a thread, the slices added in their order. `stride`: from slice to slice
__device__ __forceinline__ float4 add_slices(const float* src, int splits, int64_t stride)
{
    float4 s = __ldcs(reinterpret_cast<const float4*>(src));
    for (int q = 1; q < splits; ++q) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(src + q * stride));
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    return s;
}

template <FpEnd END>
__global__ void __launch_bounds__(256)
    k_fp_join(const float* __restrict__ P, int splits, int64_t stride, int pitch, const __grid_constant__ FpGemmArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    const int quads = pitch / 4, M = a.M, N = a.N;
    const FpEpilogue& e = a.e;
    const bool half = END == FpEnd::Grad && blockIdx.y;
    if (half) P += (int64_t)M * pitch;
    void* const y = half ? a.x.y2 : e.y;
    const int64_t ldy = half ? a.x.ldy2 : e.ldy;
    const int64_t n = (int64_t)M * quads;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = i / quads;
        const int c = (int)(i - r * quads) * 4;
        const float4 s = add_slices(P + r * pitch + c, splits, stride);
        const float v[4] = {s.x, s.y, s.z, s.w};
        if (END == FpEnd::Linear) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < N) fp_finish(e, r, c + j, v[j]);
        } else if (END == FpEnd::Gated) {
            const float4 t = add_slices(P + (int64_t)M * pitch + r * pitch + c, splits, stride);
            const float u[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < N) fp_finish_gated(e, a.x, r, c + j, v[j], u[j]);
        } else if (END == FpEnd::DLogits) {
            SlopeRow row;
            row.load(a.x, M, (int)r, c == 0 && a.x.first == 0, a.err);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < N) store_typed(e.y, e.type, r * e.ldy + c + j, row.at(v[j], c + j));
        } else {
            const float alpha = a.x.alpha ? *a.x.alpha : 1.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < N) {
                    float sum = v[j] * alpha;
                    if (a.x.acc) sum += a.x.acc[r * a.x.ldacc + c + j];
                    store_typed(y, e.out_type, r * ldy + c + j, sum);
                }
        }
    }
}

// A block to a row: its sums' largest, sum of exponentials and target's
__global__ void __launch_bounds__(256)
    k_fp_join_loss(const float* __restrict__ P, int splits, int64_t stride, int pitch, const __grid_constant__ FpGemmArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float ms[8], ss[8];
    const int64_t r = blockIdx.x;
    const int target = a.x.targets[r];
    float m = -INFINITY, s = 0.0f;
    for (int c = threadIdx.x * 4; c < a.N; c += blockDim.x * 4) {
        const float4 q = add_slices(P + r * pitch + c, splits, stride);
        const float v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (c + j >= a.N) break;
            if (c + j == target) a.x.hit[r] = v[j];
            fp_softmax_add(m, s, v[j], 1.0f);
        }
    }
    fp_softmax_warp(m, s);
    if ((threadIdx.x & 31) == 0) {
        ms[threadIdx.x >> 5] = m;
        ss[threadIdx.x >> 5] = s;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) fp_softmax_add(m, s, ms[w], ss[w]);
        a.x.part[r] = make_float2(m, s);
    }
}

// ------------------------------------------------------------------ host

struct FpPlan {
    bool pair;
    int bn, splits, kb_per_split;
};

// Which kernel, tile width and number of K slices take the least estimated time. An SM takes
// operands from L2 at about 100 KB a us (8192 x 4096 x 4096: a K block of a 256-column pair's tile is
// 32 KB an SM and took 0.32 us), a K block of products takes at least 0.27 us for 256 columns,
// and a block's loads and their waits about 0.12; a join takes 2.5 us and the slices' sums pass
// through memory at 4 TB/s. It orders the measured choices (us): 8192 x 4096 x 4096 142 with
// 256 columns, 185 with 160; 2048 x 4096 x 4096 40 with 224, 53 with 256; 512 x 4096 x 4096 23 in
// 128 x 128 tiles, 22 in pairs of 128 columns; 33 x 6080 x 5824 27 whole, 15 in three slices.
// The gated layer's tiles have two sums to a result column (their widths are multiples of 64, so that
// both of a row quarter's epilogue warps have columns); a result in halves has its row tiles twice.
static FpPlan fp_plan(int M, int N, int K, bool b_mn, FpEnd end = FpEnd::Linear, int halves = 1)
{
    const bool gated = end == FpEnd::Gated;
    const int sums = gated ? 2 : 1;              // of a result column
    const int num_kb = (K + 63) / 64, sms = num_sms(), pairs = sms / 2;
    FpPlan best{};
    double best_us = 1e30;
    // `tiles` tiles on `workers` SMs or pairs, whole and in up to 16 slices of at least four K blocks
    auto consider = [&](bool pair, int bn, int64_t tiles, int workers, double kb_us, double fixed) {
        for (int s = 1; s <= 16 && (s == 1 || num_kb / s >= 4); ++s) {
            const int per = (num_kb + s - 1) / s;
            if ((num_kb + per - 1) / per != s) continue;
            const double join = s > 1 ? 2.5 + 2.0 * s * M * N * 4 * sums * halves / 4e6 : 0;
            const double us = fixed + (double)((tiles * s + workers - 1) / workers) * per * kb_us + join;
            if (us < best_us) {
                best_us = us;
                best = FpPlan{pair, bn, s, per};
            }
        }
    };
    if (M > 128 && N * sums > 64)
        for (int bn = 256; bn >= 128; bn -= 32 * sums) {
            const int cols = bn / sums;
            const int64_t tiles = (int64_t)((M + 255) / 256) * halves * ((N + cols - 1) / cols);
            const int loaded = b_mn ? (bn + 127) / 128 * 128 : bn;
            const double kb_us = std::max(0.27 * bn / 256, (16.0 + loaded / 16.0) / 100);
            consider(true, bn, tiles, pairs, kb_us, 3);
        }
    const int64_t row_tiles = (int64_t)((M + 127) / 128) * halves;
    const double a_kb = 16.0 * std::min(M, 128) / 128;
    for (int bn = 128; bn >= 64 * sums; bn -= 64) {
        const int cols = bn / sums;
        const int64_t tiles = row_tiles * ((N + cols - 1) / cols);
        const double kb_us = std::max(0.12, (a_kb + bn / 8.0) / 100);
        consider(false, bn, tiles, sms, kb_us, 4);
    }
    return best;
}

// planes of sums that a slice leaves
static int planes(FpEnd end, int halves) { return end == FpEnd::Gated ? 2 : halves; }

static size_t plan_bytes(const FpPlan& p, int M, int N, FpEnd end, int halves)
{
    return p.splits > 1 ? align256((size_t)p.splits * planes(end, halves) * M * pad4(N) * sizeof(float)) : 0;
}

size_t fp_gemm_ws_bytes(int M, int N, int K, bool b_mn, FpEnd end, int halves, int plan_n)
{
    return plan_bytes(fp_plan(M, plan_n ? plan_n : N, K, b_mn, end, halves), M, N, end, halves);
}

int fp_loss_parts(int M, int N, int K)
{
    const FpPlan p = fp_plan(M, N, K, false, FpEnd::Loss);
    return p.splits > 1 ? 0 : 2 * ((N + p.bn - 1) / p.bn);     // (two warps to a tile's row)
}

// 2-D box map over a row-major tensor of 16-bit or 32-bit elements: rows of 128 bytes with the
// 128-byte swizzle, or of 64 bytes with the 64-byte one
static int box_map(CUtensorMap* map, void* p, bool wide, int64_t rows, int64_t cols, int64_t ld, int box_rows,
                   int row_bytes = 128)
{
    auto enc = get_encode();
    if (!enc) return set_error(ITO_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
    const int size = wide ? 4 : 2;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld * size};
    cuuint32_t box[2] = {(cuuint32_t)(row_bytes / size), (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, wide ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, p, dims,
                           strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ITO_OK : set_error(ITO_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

// whether TMA can address the rows: 16-byte aligned base and row stride (a single row's stride is free)
static bool rows_aligned(const void* p, int64_t ld, int size, int64_t rows)
{
    return aligned_to(p, 16) && (ld * size) % 16 == 0 && ld > 0 && (rows == 1 || ld * size < (int64_t(1) << 40));
}

// `kern` may have `bytes` of shared memory on the current device.
template <typename K>
static cudaError_t allow_smem(K kern, int bytes, OnEachDevice* set)
{
    int device = 0;
    const cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    return set->run(device, [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
}

// Pairs that run at the same time: a figure of the kernel and this part, the same on each device of it.
template <int PROBLEMS, FpEnd END>
static int max_pairs()
{
    static std::atomic<int> most{0};
    static OnEachDevice ready;
    const auto kern = k_fp_gemm_pair<PROBLEMS, END>;
    if (allow_smem(kern, FpPairCfg::SMEM_BYTES, &ready) != cudaSuccess) return 0;
    if (most) return most;
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
    if (cudaOccupancyMaxActiveClusters(&got, kern, &q) == cudaSuccess && got > 0) most = got;
    return most;
}

static int halves_of(const FpProduct& c) { return c.a_half ? 2 : 1; }

template <int BN, FpEnd END>
static int launch_single(const FpProblem& q, cudaStream_t s)
{
    static OnEachDevice ready;
    if (allow_smem(k_fp_gemm<BN, END>, FpCfg<BN>::SMEM_BYTES, &ready) != cudaSuccess)
        return set_error(ITO_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(cudaGetLastError()));
    const FpGemmArgs& a = q.a;
    const int64_t items = (int64_t)((a.M + 127) / 128) * a.halves * ((a.N + a.cols - 1) / a.cols) * a.splits;
    const int grid = items < num_sms() ? (int)items : num_sms();
    launch_pdl(k_fp_gemm<BN, END>, grid, FpCfg<BN>::THREADS, FpCfg<BN>::SMEM_BYTES, s, q);
    return launch_status("linear product");
}

// the arguments and tensor maps that both kernels take
static int fill_problem(FpProblem* q, const FpProduct& c, const FpPlan& p, void* ws)
{
    const FpEpilogue& e = c.e;
    const bool gated = c.end == FpEnd::Gated;
    FpGemmArgs& a = q->a;
    a.e = e;
    a.x = c.x;
    a.M = c.M;
    a.N = c.N;
    a.K = c.K;
    a.a_mn = c.A.mn;
    a.b_mn = c.B.mn;
    a.group = 16;
    a.bn = p.bn;
    a.cols = gated ? p.bn / 2 : p.bn;
    a.splits = p.splits;
    a.kb_per_split = p.kb_per_split;
    a.halves = halves_of(c);
    a.a_half = c.a_half;
    a.kb_half = c.k_half / 64;
    a.err = device_error_word();
    if (!a.err) return set_error(ITO_ERR_CUDA, "device error word unavailable");
    const bool wide = e.out_type == ITO_F32;
    const int out = wide ? 4 : 2;
    a.y_tma = e.y && rows_aligned(e.y, e.ldy, out, c.M);
    a.z_tma = e.z && rows_aligned(e.z, e.ldz, 2, c.M);
    void* const y2 = gated ? c.x.z2 : c.x.y2;
    const int64_t ldy2 = gated ? c.x.ldz2 : c.x.ldy2;
    a.y2_tma = a.z2_tma = y2 && rows_aligned(y2, ldy2, out, c.M);
    a.b_vec = aligned_to(e.bias, 16);
    a.b2_vec = aligned_to(c.x.bias2, 16);
    a.r_vec = c.x.acc ? rows_aligned(c.x.acc, c.x.ldacc, 4, c.M)
                      : e.residual && rows_aligned(e.residual, e.ldr, out, c.M);
    a.idesc = fp_idesc(p.pair ? 256 : 128, p.bn, c.A.mn, c.B.mn, e.type == ITO_BF16);
    const int64_t rows = c.a_half ? (int64_t)c.a_half + c.M : c.M;
    int r = box_map(&q->A, const_cast<void*>(c.A.p), false, c.A.mn ? c.K : rows, c.A.mn ? rows : c.K, c.A.ld,
                    c.A.mn ? 64 : 128);
    // (rows of a B in two halves end before its last K block does: those beyond come as 0)
    const int64_t k_rows = c.k_half ? c.k_rows : c.K;
    const int box = c.B.mn ? 64 : p.pair || gated ? p.bn / 2 : p.bn;
    if (!r)
        r = box_map(&q->B, const_cast<void*>(c.B.p), false, c.B.mn ? k_rows : c.N, c.B.mn ? c.N : c.K, c.B.ld, box);
    if (!r && c.B2.p)
        r = box_map(&q->B2, const_cast<void*>(c.B2.p), false, c.B.mn ? k_rows : c.N, c.B.mn ? c.N : c.K, c.B2.ld, box);
    if (!r && a.y_tma) r = box_map(&q->Y, e.y, wide, c.M, c.N, e.ldy, 32, 64);
    if (!r && a.z_tma) r = box_map(&q->Z, e.z, false, c.M, c.N, e.ldz, 32, 64);
    if (!r && a.y2_tma) r = box_map(&q->Y2, y2, wide, c.M, c.N, ldy2, 32, 64);
    if (!r && p.splits > 1) {
        // the slices' sums [splits][planes][M][pitch]
        const int64_t pitch = pad4(c.N);
        auto enc = get_encode();
        cuuint64_t dims[3] = {(cuuint64_t)pitch, (cuuint64_t)c.M, (cuuint64_t)p.splits * planes(c.end, a.halves)};
        cuuint64_t strides[2] = {(cuuint64_t)pitch * 4, (cuuint64_t)pitch * c.M * 4};
        cuuint32_t box3[3] = {16, 32, 1};
        cuuint32_t estr[3] = {1, 1, 1};
        const CUresult cr = enc(&q->S, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, ws, dims, strides, box3, estr,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                                CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (cr != CUDA_SUCCESS) r = set_error(ITO_ERR_CUDA, "cuTensorMapEncodeTiled (partials) failed (%d)", (int)cr);
    }
    return r;
}

template <FpEnd END>
static int run_join(const FpGemmArgs& a, const void* ws, cudaStream_t s)
{
    const int64_t pitch = pad4(a.N), plane = pitch * a.M, stride = plane * planes(END, a.halves);
    const float* P = static_cast<const float*>(ws);
    if constexpr (END == FpEnd::Loss) {
        launch_pdl(k_fp_join_loss, a.M, 256, 0, s, P, a.splits, stride, (int)pitch, a);
        return launch_status("linear join");
    } else {
        launch_pdl(k_fp_join<END>, dim3(launch_grid_blocks((int64_t)a.M * (pitch / 4), 256), a.halves), 256, 0, s, P,
                   a.splits, stride, (int)pitch, a);
        return launch_status("linear join");
    }
}

static int pair_items(const FpProblem& q)
{
    return ((q.a.M + 255) / 256) * q.a.halves * ((q.a.N + q.a.cols - 1) / q.a.cols) * q.a.splits;
}

template <int PROBLEMS, FpEnd END>
static int launch_pairs(FpPairWork<PROBLEMS>& w, cudaStream_t s)
{
    const int most = max_pairs<PROBLEMS, END>();
    if (!most) return set_error(ITO_ERR_CUDA, "no CTA pair fits on this device");
    const int items = w.items[0] + w.items[1], pairs = items < most ? items : most;
    w.rest = w.gap = 0;
    if (PROBLEMS == 2) {
        w.rest = w.items[0] % pairs;
        // K blocks tell an item's time (both problems' tiles have the same width or nearly), where it is above its
        // epilogue's, about that of 10 K blocks (a weight gradient of 333 rows has 6; Linear keeps its order)
        const int least = END == FpEnd::Grad ? 10 : 1;
        if (w.rest) w.gap = std::max(w.p[0].a.kb_per_split, least) / std::max(w.p[PROBLEMS - 1].a.kb_per_split, least);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_fp_gemm_pair<PROBLEMS, END>, w);
    return e == cudaSuccess ? ITO_OK : set_error(ITO_ERR_CUDA, "linear product launch: %s", cudaGetErrorString(e));
}

template <FpEnd END>
static int run_products(const FpProduct* c, int n, void* ws, cudaStream_t s)
{
    FpPlan p[2];
    FpProblem q[2];
    void* at[2];
    for (int i = 0; i < n; ++i) {
        p[i] = fp_plan(c[i].M, c[i].plan_n ? c[i].plan_n : c[i].N, c[i].K, c[i].B.mn, END, halves_of(c[i]));
        at[i] = ws;
        ws = static_cast<char*>(ws) + plan_bytes(p[i], c[i].M, c[i].N, END, halves_of(c[i]));
        memset(&q[i], 0, sizeof(q[i]));
        const int r = fill_problem(&q[i], c[i], p[i], at[i]);
        if (r) return r;
    }
    constexpr bool TWO = END == FpEnd::Linear || END == FpEnd::Grad;
    const bool both = TWO && n == 2 && p[0].pair && p[1].pair;
    if constexpr (TWO) {
        if (both) {
            FpPairWork<2> w;
            const int first = p[0].kb_per_split >= p[1].kb_per_split ? 0 : 1;
            for (int i = 0; i < 2; ++i) {
                w.p[i] = q[first ^ i];
                w.items[i] = pair_items(w.p[i]);
            }
            const int r = launch_pairs<2, END>(w, s);
            if (r) return r;
        }
    }
    for (int i = 0; i < n; ++i) {
        int r = ITO_OK;
        if (!both && p[i].pair) {
            FpPairWork<1> w;
            w.p[0] = q[i];
            w.items[0] = pair_items(q[i]);
            w.items[1] = 0;
            r = launch_pairs<1, END>(w, s);
        } else if (!both) {
            if (END == FpEnd::Gated || p[i].bn == 128) r = launch_single<128, END>(q[i], s);
            else if constexpr (END != FpEnd::Gated) r = launch_single<64, END>(q[i], s);
        }
        if (!r && p[i].splits > 1) r = run_join<END>(q[i].a, at[i], s);
        if (r) return r;
    }
    return ITO_OK;
}

int fp_gemm(const FpProduct* c, int n, void* ws, cudaStream_t s)
{
    switch (c[0].end) {
    case FpEnd::Gated: return run_products<FpEnd::Gated>(c, n, ws, s);
    case FpEnd::Loss: return run_products<FpEnd::Loss>(c, n, ws, s);
    case FpEnd::DLogits: return run_products<FpEnd::DLogits>(c, n, ws, s);
    case FpEnd::Grad: return run_products<FpEnd::Grad>(c, n, ws, s);
    default: return run_products<FpEnd::Linear>(c, n, ws, s);
    }
}

}  // namespace ito
