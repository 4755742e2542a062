// The gradients of a linear product of a few rows, with one weight or two:
//
//   dx[b][c] = sum_v g[b][v] W[v][c]        dW[v][c] = sum_b g[b][v] x[b][c]        b < 16
//
// dx reads every weight once and dW writes as much once; there is little else to do, and memory bounds both. In tiles of
// the tensor cores' kernels, of 128 rows, most of each product is of rows that do not exist, and a dW's many
// short products leave at 0.6 of the copy rate. Here (8 rows, two weights of 32768 x 4096, bf16) dx takes 88 us, 6.1 TB/s
// of W, dW 79 (6.8 TB/s) and both 176, 0.90 of the copy rate; in tiles 87, 123 and 223. Weights of 32767 x 2051 (rows
// at any alignment) take 68, 90 and 157 instead of 131, 150 and 303, copies of the weights included.
//
// One launch has the blocks of both, dx's first. (Mixed evenly, so that reads and writes go on together, both took 217 instead of 189.)
//
// The products are m16n8k16 ones on pairs of rows (of W, or of x). A lane has eight consecutive columns of each of four
// rows; byte permutes make of them the operands of eight products, the j-th of which takes column j of each
// lane's eight. The eights of lane group g are the g / 2 + 4 (g % 2)-th of 64 columns: a dW's two columns of a
// lane, over the eight products, are then two runs of eight consecutive ones, and a quad's runs are neighbours (64
// bytes of a 16-bit row).
#include "ito_fp_rows.cuh"

namespace ito {

constexpr int kFgThreads = 256, kFgWarps = kFgThreads / 32;
constexpr int kFgColumns = 64;       // of a warp's products
constexpr int kFgRows = 16;          // of the weights, taken at a time: a chunk

struct FewGrad {
    FpFewGrad p;
    int groups;                      // of 64 columns
    int chunks;                      // of a weight
    int log_wide;                    // of dx: warps of a block side by side, the others take turns along the chunks
    int wide_groups, splits, dx_chunks, dx_blocks;       // (splits, strips: of each weight)
    int strips, dw_chunks;
    int shares;                      // splits of all weights
    float* sums;                     // [shares][B][pitch]
    int64_t pitch;
    int dw_vec;
};

template <bool ALREADY>
__device__ __forceinline__ const uint16_t* aligned16(const uint16_t* p)
{
    return ALREADY ? p : reinterpret_cast<const uint16_t*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15));
}

// word j / 2 of a row's eight and of another's -> (column j of the one, of the other)
__device__ __forceinline__ uint32_t column_pair(const uint4& lo, const uint4& hi, int j)
{
    const uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
    return __byte_perm(a[j >> 1], b[j >> 1], j & 1 ? 0x7632 : 0x5410);
}

// an 8 x 8 matrix of 16-bit elements over a warp, transposed
__device__ __forceinline__ uint32_t transposed(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// 16 bytes of W, or its first `bytes` and zeros, to shared memory in the background (a row's 128 bytes come with the
// next 128: 2 x 32768 x 4096 97 us instead of 101); eight bytes of g, or zeros
__device__ __forceinline__ void copy16_async(void* dst, const void* src, int bytes)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy8_async(void* dst, const void* src, bool in)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 8 : 0)
                 : "memory");
}

// A chunk on its way through shared memory: 64 columns of 16 rows of W, as the aligned 16 bytes that hold them (nine where
// rows start anywhere), and each lane's g of four rows for NT eights of tokens
template <int NT, bool VEC>
struct DxStage {
    uint4 w[kFgRows][VEC ? 8 : 9];
    uint2 f[NT][32];
};
constexpr int kFgStages = 4;

// dx: a block takes a share of a weight's chunks; its warps lie side by side over 64 columns each, or take turns along
// the chunks (then their sums meet in shared memory, in their order). The shares' sums meet in k_fp_few_join. Here the
// 16 x 8 operand is g's, eight tokens, and the 16 x 16 one two columns of each lane's eight. (With the chunks loaded to
// registers, few of them at a time, 200 us instead of 88 in the case above.)
template <int NT, bool VEC>
__device__ __forceinline__ void few_dx(const FewGrad& a, int block, uint8_t* smem)
{
    const FpFewGrad& p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int wide = 1 << a.log_wide, turns = kFgWarps >> a.log_wide, turn = warp >> a.log_wide;
    const int group = block % a.wide_groups * wide + (warp & (wide - 1)), split = block / a.wide_groups;
    const int place = (g >> 1) + 4 * (g & 1);
    const int seg = split >= a.splits;
    const int lo = (split - (seg ? a.splits : 0)) * a.dx_chunks, hi = min(a.chunks, lo + a.dx_chunks);
    auto* const ring = reinterpret_cast<DxStage<NT, VEC>*>(smem) + warp * kFgStages;
    const int c0 = group * kFgColumns;
    const uint16_t* const W = p.W[seg];
    const int64_t ld = p.ldw[seg];
    const uint16_t* const end = W + (p.V - 1) * ld + p.D;
    // this lane's four rows of a chunk are consecutive ones (the order of a sum is free); from the place of the next
    // chunk's that is copied, and of the one that is multiplied
    const int64_t step = (int64_t)turns * kFgRows * ld;
    const uint16_t* next = W + (int64_t)((lo + turn) * kFgRows + 4 * t) * ld + c0;
    const uint16_t* here = next;
    const uint16_t* fg[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        fg[n] = p.g[seg] + (8 * n + g < p.B ? 8 * n + g : 0) * p.ldg + (lo + turn) * kFgRows + 4 * t;
    auto fetch = [&](int chunk, DxStage<NT, VEC>& to) {
        const int v0 = chunk * kFgRows;
        // All that is read lies in W but for its first rows and its last (an aligned 16 bytes begin seven elements
        // before the 64 and end as many behind them at most).
        if (c0 < p.D && chunk < hi) {
            if (VEC ? v0 + kFgRows <= p.V && c0 + kFgColumns <= p.D : v0 > 0 && v0 + 2 * kFgRows <= p.V && ld >= 8) {
#pragma unroll
                for (int r = 0; r < 4; ++r) copy16_async(&to.w[4 * t + r][g], aligned16<VEC>(next + r * ld) + 8 * g, 16);
                if (!VEC && g < 4)
                    copy16_async(&to.w[4 * t + g][VEC ? 0 : 8], aligned16<VEC>(next + g * ld) + kFgColumns, 16);
            } else {
                auto copy = [&](int r, int at) {         // the bytes that exist, or zeros
                    const uint16_t* from = aligned16<VEC>(next + r * ld) + 8 * at;
                    int bytes = 16;
                    if (v0 + 4 * t + r >= p.V || from < W || end <= from) bytes = 0;
                    else if (end - from < 8) bytes = (int)(end - from) * 2;
                    copy16_async(&to.w[4 * t + r][at], bytes ? from : aligned16<false>(W), bytes);
                };
                for (int r = 0; r < 4; ++r) copy(r, g);
                if (!VEC && g < 4) copy(g, 8);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const bool in = 8 * n + g < p.B && v0 + 4 * t < p.V;
                copy8_async(&to.f[n][lane], in ? fg[n] : p.g[seg], in);
                fg[n] += turns * kFgRows;
            }
        }
        next += step;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // eight columns of the lane's r-th row
    auto get = [&](const DxStage<NT, VEC>& from, int v, int r) {
        if constexpr (VEC) {
            return from.w[4 * t + r][place];
        } else {
            const uint16_t* const at = here + r * ld + 8 * place;
            if (v < kFgRows && aligned16<false>(at) < W && v < p.V) return load_eight(at, 0, p.D, false);
            const uint32_t* const words = reinterpret_cast<const uint32_t*>(&from.w[4 * t + r][place]) +
                                          (reinterpret_cast<uintptr_t>(at) >> 2 & 3);
            Eight16 e;
#pragma unroll
            for (int i = 0; i < 5; ++i) e.w[i] = words[i];
            return e.get(at);
        }
    };
    float s[NT][4][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][j][i] = 0.0f;
#pragma unroll
    for (int i = 0; i < kFgStages - 1; ++i) fetch(lo + turn + i * turns, ring[i]);
    int stage = 0;
    for (int chunk = lo + turn; chunk < hi && c0 < p.D; chunk += turns) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kFgStages - 2) : "memory");
        __syncwarp();                                // this stage is there for all lanes, the last one read by all
        fetch(chunk + (kFgStages - 1) * turns, ring[(stage + kFgStages - 1) % kFgStages]);
        const DxStage<NT, VEC>& from = ring[stage];
        stage = (stage + 1) % kFgStages;
        const int v = chunk * kFgRows + 4 * t;
        uint4 w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = get(from, v + r, r);
        here += step;
        uint2 f[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            f[n] = from.f[n][lane];
            if (v + 4 > p.V) {                       // (what a row of g holds from V on does not count)
                if (v + 1 >= p.V) f[n].x &= 0xFFFFu;
                if (v + 2 >= p.V) f[n].y = 0u;
                if (v + 3 >= p.V) f[n].y &= 0xFFFFu;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t a0 = column_pair(w[0], w[1], 2 * j), a1 = column_pair(w[0], w[1], 2 * j + 1);
            const uint32_t a2 = column_pair(w[2], w[3], 2 * j), a3 = column_pair(w[2], w[3], 2 * j + 1);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16816(p.type, s[n][j], a0, a1, a2, a3, f[n].x, f[n].y);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    float(*const part)[8][kFgColumns + 1] = reinterpret_cast<float(*)[8][kFgColumns + 1]>(smem);
    const float alpha = a.shares == 1 && p.alpha ? *p.alpha : 1.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[warp][2 * t + (i & 1)][8 * place + 2 * j + (i >> 1)] = s[n][j][i];
        __syncthreads();
        for (int i = threadIdx.x; i < 8 * kFgColumns << a.log_wide; i += kFgThreads) {
            const int k = i % kFgColumns, j = i / kFgColumns & (wide - 1), of = i / kFgColumns >> a.log_wide;
            const int b = 8 * n + of, col = (block % a.wide_groups * wide + j) * kFgColumns + k;
            if (b >= p.B || col >= p.D) continue;
            float v = part[j][of][k];
            for (int w = 1; w < turns; ++w) v += part[j + (w << a.log_wide)][of][k];
            if (a.shares > 1) a.sums[((int64_t)split * p.B + b) * a.pitch + col] = v;
            else store_typed(p.dx, p.type, b * p.lddx + col, v * alpha);
        }
    }
}

// Eight columns of row b of x (0 beyond it)
template <bool VEC>
__device__ __forceinline__ uint4 x_eight(const FpFewGrad& p, int b, int c)
{
    if (b >= p.B || c >= p.D) return make_uint4(0u, 0u, 0u, 0u);
    const uint16_t* const at = p.x + b * p.ldx + c;
    if (!VEC && c + 8 <= p.D && Eight16::whole(at, p.x, p.x + (p.B - 1) * p.ldx + p.D)) {
        Eight16 e;
        e.load(at);
        return e.get(at);
    }
    return load_eight(at, 0, p.D - c, VEC);
}

// Rows of 128 bytes in shared memory, as a warp writes them where result rows do not start on 16-byte boundaries
struct DwRows {
    uint32_t w[kFgRows][36];         // (16 bytes more: rows in different banks)
};

// dW: a warp keeps 64 columns of x and goes through a strip of chunks
template <bool VEC>
__device__ __forceinline__ void few_dw(const FewGrad& a, int64_t unit, DwRows& rows)
{
    const FpFewGrad& p = a.p;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int group = (int)(unit % a.groups);
    int strip = (int)(unit / a.groups);
    const int seg = strip >= a.strips;
    if (seg) strip -= a.strips;
    if (strip >= a.strips || (seg && !p.g[1])) return;
    const uint16_t* const gs = p.g[seg];
    void* const out = p.dW[seg];
    const int64_t ld = p.lddw[seg];
    const int c0 = group * kFgColumns;
    uint32_t x[8][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int b = 8 * h + 2 * t, c = c0 + 8 * ((g >> 1) + 4 * (g & 1));
        const uint4 lo = x_eight<VEC>(p, b, c), hi = x_eight<VEC>(p, b + 1, c);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j][h] = column_pair(lo, hi, j);
    }
    const float alpha = p.alpha ? *p.alpha : 1.0f;
    const int lo = strip * a.dw_chunks, hi = min(a.chunks, lo + a.dw_chunks);
    // g of a chunk, [token][row of the weight]: the transposed products' first operand
    auto load = [&](int chunk, uint32_t (&f)[4]) {
        const uint16_t* const from = gs + chunk * kFgRows + 2 * t;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int b = 8 * h + g;
            f[2 * h] = f[2 * h + 1] = 0u;
            if (chunk < hi && b < p.B) {
                const uint16_t* const row = from + b * p.ldg;
                f[2 * h] = __ldg(reinterpret_cast<const uint32_t*>(row));
                f[2 * h + 1] = __ldg(reinterpret_cast<const uint32_t*>(row + 8));
            }
        }
    };
    uint32_t f[4];
    load(lo, f);
#pragma unroll 1
    for (int chunk = lo; chunk < hi; ++chunk) {
        uint32_t next[4];
        load(chunk + 1, next);
        float s[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = transposed(f[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) mma_16816(p.type, s[j], f[0], f[1], f[2], f[3], x[j][0], x[j][1]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i] *= alpha;
        const int v0 = chunk * kFgRows;
        const bool wide = p.out_type == ITO_F32;
        if (a.dw_vec) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int v = v0 + g + 8 * h, c = c0 + 32 * i + 8 * t, k = 2 * h + i;
                    if (v >= p.V || c >= p.D) continue;
                    if (wide) {
                        float4* const to = reinterpret_cast<float4*>(static_cast<float*>(out) + v * ld + c);
                        to[0] = make_float4(s[0][k], s[1][k], s[2][k], s[3][k]);
                        to[1] = make_float4(s[4][k], s[5][k], s[6][k], s[7][k]);
                    } else {
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + v * ld + c) =
                            make_uint4(pack16(p.type, s[0][k], s[1][k]), pack16(p.type, s[2][k], s[3][k]),
                                       pack16(p.type, s[4][k], s[5][k]), pack16(p.type, s[6][k], s[7][k]));
                    }
                }
        } else if (wide) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {            // 32 columns at a time
                __syncwarp();
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 8; j += 4)
                        *reinterpret_cast<float4*>(&rows.w[g + 8 * h][8 * t + j]) =
                            make_float4(s[j][2 * h + i], s[j + 1][2 * h + i], s[j + 2][2 * h + i], s[j + 3][2 * h + i]);
                __syncwarp();
                const int c = c0 + 32 * i + lane;
#pragma unroll 4
                for (int r = 0; r < kFgRows; ++r)
                    if (v0 + r < p.V && c < p.D) static_cast<float*>(out)[(v0 + r) * ld + c] = __uint_as_float(rows.w[r][lane]);
            }
        } else {
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = 2 * h + i;
                    *reinterpret_cast<uint4*>(&rows.w[g + 8 * h][16 * i + 4 * t]) =
                        make_uint4(pack16(p.type, s[0][k], s[1][k]), pack16(p.type, s[2][k], s[3][k]),
                                   pack16(p.type, s[4][k], s[5][k]), pack16(p.type, s[6][k], s[7][k]));
                }
            __syncwarp();
            // a word of two columns to a lane; in a row that starts on an odd element the words are shifted by one, and
            // its first element is stored alone
            uint16_t* to = static_cast<uint16_t*>(out) + v0 * ld + c0;
            const int cols = min(kFgColumns, p.D - c0);
#pragma unroll 8
            for (int r = 0; r < kFgRows; ++r, to += ld) {
                const bool in = v0 + r < p.V, odd = reinterpret_cast<uintptr_t>(to) & 2;
                const int at = 2 * lane + odd;       // columns at and at + 1
                const uint32_t word = rows.w[r][lane];
                const uint32_t y = odd ? __funnelshift_r(word, rows.w[r][lane + 1], 16) : word;
                if (in && at + 1 < cols) *reinterpret_cast<uint32_t*>(to + at) = y;
                if (in && at + 1 == cols) to[at] = (uint16_t)y;
                if (in && odd && lane == 0) to[0] = (uint16_t)word;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = next[i];
    }
}

template <int NT, bool VEC>
constexpr int kFgSmem = std::max<int>(sizeof(DxStage<NT, VEC>) * kFgStages * kFgWarps,
                                      std::max(sizeof(float) * kFgWarps * 8 * (kFgColumns + 1), sizeof(DwRows) * kFgWarps));

template <int NT, bool VEC>
__global__ void __launch_bounds__(kFgThreads, 2) k_fp_few_grad(const __grid_constant__ FewGrad a)
{
    extern __shared__ __align__(16) uint8_t few_smem[];
    griddep_wait();
    griddep_launch_dependents();
    const int block = (int)blockIdx.x - a.dx_blocks, warp = threadIdx.x >> 5;
    if (block < 0) few_dx<NT, VEC>(a, blockIdx.x, few_smem);
    else few_dw<VEC>(a, (int64_t)block * kFgWarps + warp, reinterpret_cast<DwRows*>(few_smem)[warp]);
}

// dx from the shares' sums: a block takes 128 columns of a row, four to a thread, and eight threads a share each of the
// sums, which are added in the shares' order
__global__ void __launch_bounds__(kFgThreads) k_fp_few_join(const __grid_constant__ FewGrad a)
{
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float4 part[8][32];
    const FpFewGrad& p = a.p;
    const int blocks = (int)((a.pitch + 127) / 128);
    const int b = blockIdx.x / blocks, quad = threadIdx.x & 31, share = threadIdx.x >> 5;
    const int64_t c = (int64_t)(blockIdx.x % blocks) * 128 + quad * 4;
    const int per = (a.shares + 7) / 8, q0 = share * per, q1 = min(a.shares, q0 + per);
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < p.D) {
#pragma unroll 8
        for (int q = q0; q < q1; ++q) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(a.sums + ((int64_t)q * p.B + b) * a.pitch + c));
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
    }
    part[share][quad] = s;
    __syncthreads();
    if (threadIdx.x >= 128) return;
    const int64_t col = (int64_t)(blockIdx.x % blocks) * 128 + threadIdx.x;
    if (col >= p.D) return;
    float v = 0.0f;
    for (int w = 0; w < 8; ++w) v += reinterpret_cast<const float*>(&part[w][0])[threadIdx.x];
    store_typed(p.dx, p.type, b * p.lddx + col, p.alpha ? v * *p.alpha : v);
}

// ------------------------------------------------------------------------ host

static FewGrad few_plan(int B, int V, int D, int segs)
{
    FewGrad a{};
    const int sms = num_sms();
    a.groups = (D + kFgColumns - 1) / kFgColumns;
    a.chunks = (V + kFgRows - 1) / kFgRows;
    // Warps side by side read longer runs of a row, those that take turns leave fewer sums to join: four side by side
    // where a warp has a dozen chunks and more (us of 1, 2, 4, 8: dx of 8 rows, 2 x 32768 x 4096 97, 97, 89, 86; all of 16
    // rows, 2 x 8192 x 2048 32, 33, 34, 36 and of 8 rows, 2 x 4096 x 1024 10, 11, 12, 13). Two blocks to an SM at most (more
    // have a last round of few: the first of these in 320 blocks 110); two chunks to a warp at least.
    const int64_t each = (int64_t)a.groups * a.chunks * segs / (2 * sms * kFgWarps);
    if (each >= 12)
        while (a.log_wide < 2 && (1 << a.log_wide) < a.groups) ++a.log_wide;
    a.wide_groups = (a.groups + (1 << a.log_wide) - 1) >> a.log_wide;
    const int splits = std::max(1, std::min(2 * sms / (a.wide_groups * segs), a.chunks / (2 * kFgWarps >> a.log_wide)));
    a.dx_chunks = (a.chunks + splits - 1) / splits;
    a.splits = (a.chunks + a.dx_chunks - 1) / a.dx_chunks;
    a.shares = a.splits * segs;
    a.pitch = (int64_t)a.groups * kFgColumns;
    const int strips = std::max(1, std::min((2 * sms * kFgWarps + a.groups * segs - 1) / (a.groups * segs), a.chunks / 4));
    a.dw_chunks = (a.chunks + strips - 1) / strips;
    a.strips = (a.chunks + a.dw_chunks - 1) / a.dw_chunks;
    return a;
}

// us, both gradients of two weights, as here : in tiles: 16 rows, 8192 x 2048 34 : 40, 32768 x 4096 190 : 224, 8 rows, 4096 x
// 1024 10 : 17; 32 rows (with four eights of tokens) 8192 x 2048 59 : 40.
bool fp_few_grad_rows(int B) { return B <= 16; }

size_t fp_few_grad_ws_bytes(int B, int V, int D, int segs)
{
    const FewGrad a = few_plan(B, V, D, segs);
    return a.shares > 1 ? align256((size_t)a.shares * B * a.pitch * sizeof(float)) : 0;
}

template <int NT, bool VEC>
static int few_launch(const FewGrad& a, int grid, cudaStream_t s)
{
    static OnEachDevice ready;
    const auto kern = k_fp_few_grad<NT, VEC>;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess)
        e = ready.run(device, [&] {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFgSmem<NT, VEC>);
        });
    if (e == cudaSuccess) e = launch_pdl(kern, grid, kFgThreads, kFgSmem<NT, VEC>, s, a);
    return e == cudaSuccess ? ITO_OK : set_error(ITO_ERR_CUDA, "gradients of a few rows: %s", cudaGetErrorString(e));
}

int fp_few_grad(const FpFewGrad& p, void* ws, cudaStream_t s)
{
    const int segs = p.g[1] ? 2 : 1;
    FewGrad a = few_plan(p.B, p.V, p.D, segs);
    a.p = p;
    a.sums = static_cast<float*>(ws);
    a.dx_blocks = p.dx ? a.wide_groups * a.shares : 0;
    bool vec = p.D % 8 == 0;
    a.dw_vec = p.D % 8 == 0;
    for (int i = 0; i < segs; ++i) {
        if (p.dx) vec = vec && fp_tma_rows(p.W[i], p.ldw[i], p.V, p.D);
        if (p.dW[i]) a.dw_vec = a.dw_vec && rows_vec(p.dW[i], p.lddw[i], type_bytes(p.out_type), p.V);
    }
    if (p.dW[0]) vec = vec && fp_tma_rows(p.x, p.ldx, p.B, p.D);
    const int64_t units = p.dW[0] ? (int64_t)a.groups * a.strips * segs : 0;
    const int grid = a.dx_blocks + (int)((units + kFgWarps - 1) / kFgWarps);
    int r;
    if (p.B <= 8) r = vec ? few_launch<1, true>(a, grid, s) : few_launch<1, false>(a, grid, s);
    else r = vec ? few_launch<2, true>(a, grid, s) : few_launch<2, false>(a, grid, s);
    if (r) return r;
    if (p.dx && a.shares > 1)
        launch_pdl(k_fp_few_join, p.B * (int)((a.pitch + 127) / 128), kFgThreads, 0, s, a);
    return launch_status("gradients of a few rows");
}

}  // namespace ito
