// Layer norm over the last dimension, forward and backward.
//
//   mean = sum x / n      rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)      h = (x - mean) rstd
//   y = h gamma + beta
//   a = dy gamma;  dx = rstd (a - sum(a) / n - h sum(a h) / n)
//   dgamma = sum over rows of dy h;  dbeta = sum over rows of dy
//
// The variance is taken from the centred values (a second pass over the row), not as the
// difference of two large sums. Sums are held in 32 bits.
#include <algorithm>

#include "ito_float.cuh"

namespace ito {

// A row's elements stay in registers between the passes over them: each of the row's threads
// holds VPT vectors of 16 bytes, vector i * tpr + its place. Rows of up to 32 threads' vectors
// belong to parts of a warp (tpr 1, 2, .. 32 lanes, several rows to a block, sums by shuffles);
// longer ones to a whole block, whose R rows at a time share each exchange of sums through
// shared memory and keep R * VPT loads a thread in flight. A thread's columns are the same in
// every row, so gamma, beta and the sums of dgamma and dbeta are registers too.
constexpr int kLnBlock = 256;        // threads of a block of short rows
constexpr int kLnMostThreads = 1024;

// threads of a block whose threads hold VPT vectors (ln_shape), which bounds their registers
constexpr int ln_threads(int vpt) { return vpt == 1 ? 256 : vpt == 2 ? 512 : kLnMostThreads; }
constexpr int ln_bwd_threads(int vpt) { return vpt == 1 ? 256 : 512; }

// The warp's sums of N values (a power of two) in every lane's v[0], value (lane * N) / 32: each
// exchange halves the values a lane carries, so that N sums take N + 3 or so exchanges, not 5 N.
template <int N, int M>
__device__ __forceinline__ void fold_sums(float (&v)[N])
{
    constexpr int o = 16 * M / N;
    const bool high = threadIdx.x & o;
#pragma unroll
    for (int i = 0; i < M / 2; ++i) {
        const float keep = high ? v[i + M / 2] : v[i], give = high ? v[i] : v[i + M / 2];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
    if constexpr (M > 2) fold_sums<N, M / 2>(v);
}

// Sums R values over the threads of a row: lanes of a warp (tpr <= 32) or the block. `red` holds
// two banks of R * 32 floats; the caller alternates them, so that one barrier is enough. (Eight
// warps have steps of their own: with the loops of any number the layer norm of 8192 x 4096 bf16
// took 28.4 us forward and 46.6 backward instead of 26.2 and 44.8; with 16-byte loads of the
// warps' parts and additions instead of shuffles 31.0 and 48.8.)
template <int R>
__device__ __forceinline__ void row_sums(float (&v)[R], int tpr, float* red)
{
    if (tpr <= 32) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            for (int o = tpr >> 1; o > 0; o >>= 1) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if constexpr (R > 1) fold_sums<R, R>(v);
#pragma unroll
    for (int o = 16 / R; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    if (lane % (32 / R) == 0) red[lane / (32 / R) * 32 + warp] = v[0];
    __syncthreads();
    if (warps == 8) {
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = red[r * 32 + (lane & 7)];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
#pragma unroll
            for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
        return;
    }
    int top = 2;                         // the warps' number, to the next power of two
    while (top < warps) top *= 2;
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = (lane & (top - 1)) < warps ? red[r * 32 + (lane & (top - 1))] : 0.0f;
    for (int o = top >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
}

// N weights from column c, a multiple of N (`fill` where there are none)
template <bool FULL, int N>
__device__ __forceinline__ void load_weights(const void* p, int type, int c, int n, float fill, float (&v)[N])
{
    if (FULL && p && c < n) {
        if (type == ITO_F32) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c) + i);
                v[4 * i] = f.x;
                v[4 * i + 1] = f.y;
                v[4 * i + 2] = f.z;
                v[4 * i + 3] = f.w;
            }
        } else if constexpr (N == 8) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + c));
            if (type == ITO_BF16) Vec<__nv_bfloat16>{w}.get(v);
            else Vec<__half>{w}.get(v);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = !FULL && p && c + i < n ? load_typed(p, type, c + i) : fill;
}

// FULL: rows are whole vectors on 16-byte boundaries, gamma and beta too (no element is looked at
// alone). Else a thread's elements are a row's threads apart, so that a warp's single accesses are
// still consecutive (5000 x 2500 bf16: 25 us forward and 37 backward, 41 and 75 with neighbours;
// 65536 x 30 8 and 12, 19 and 17).
template <bool FULL, int PER>
struct LnColumns {
    int tpr, at;
    __device__ __forceinline__ int first(int i) const { return FULL ? (i * tpr + at) * PER : i * PER * tpr + at; }
    __device__ __forceinline__ int step() const { return FULL ? 1 : tpr; }
    __device__ __forceinline__ int column(int i, int j) const { return first(i) + j * step(); }

    template <typename T>
    __device__ __forceinline__ void load(Vec<T>& v, const T* row, int i, int cols) const
    {
        if (FULL) v.raw = *reinterpret_cast<const uint4*>(row + first(i));
        else v.load_apart(row, first(i), tpr, cols);
    }
    template <typename T>
    __device__ __forceinline__ void store(const Vec<T>& v, T* row, int i, int cols) const
    {
        if (FULL) *reinterpret_cast<uint4*>(row + first(i)) = v.raw;
        else v.store_apart(row, first(i), tpr, cols);
    }
    __device__ __forceinline__ void weights(const void* p, int type, int i, int cols, float fill, float (&v)[PER]) const
    {
        if constexpr (FULL) {
            load_weights<true>(p, type, first(i), cols, fill, v);
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j) v[j] = p && column(i, j) < cols ? load_typed(p, type, column(i, j)) : fill;
        }
    }
};

template <typename T, int VPT, int R, bool FULL>
__global__ void __launch_bounds__(ln_threads(VPT), 1024 / ln_threads(VPT))
    k_layer_norm_fwd(const T* __restrict__ x, int64_t ldx, const void* __restrict__ gamma,
                     const void* __restrict__ beta, int w_type, int64_t rows, int cols, int tpr, float eps,
                     T* __restrict__ y, int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int PER = Vec<T>::kPer;
    __shared__ float red[2][R * 32];
    const int at = threadIdx.x % tpr, groups = blockDim.x / tpr;
    const LnColumns<FULL, PER> part{tpr, at};
    const float inv = 1.0f / (float)cols;
    const int64_t step = (int64_t)gridDim.x * groups * R;
    // every thread of the block passes the barriers of every round
    for (int64_t r0 = (int64_t)blockIdx.x * groups * R; r0 < rows; r0 += step) {
        const int64_t first = r0 + (int64_t)(threadIdx.x / tpr) * R;
        Vec<T> v[R][VPT];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (first + r < rows && part.first(i) < cols) part.load(v[r][i], x + (first + r) * ldx, i, cols);
                else v[r][i].raw = make_uint4(0u, 0u, 0u, 0u);
            }
        float mu[R], rs[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mu[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float f[PER];
                v[r][i].get(f);
#pragma unroll
                for (int j = 0; j < PER; ++j) mu[r] += f[j];
            }
        }
        row_sums<R>(mu, tpr, red[0]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mu[r] *= inv;
            rs[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float f[PER];
                v[r][i].get(f);
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const float d = (FULL ? part.first(i) : part.column(i, j)) < cols ? f[j] - mu[r] : 0.0f;
                    rs[r] += d * d;
                }
            }
        }
        row_sums<R>(rs, tpr, red[1]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            rs[r] = 1.0f / sqrtf(rs[r] * inv + eps);
            if (at == 0 && first + r < rows) {
                if (mean) mean[first + r] = mu[r];
                if (rstd) rstd[first + r] = rs[r];
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (part.first(i) >= cols) continue;
            float g[PER], b[PER];
            part.weights(gamma, w_type, i, cols, 1.0f, g);
            part.weights(beta, w_type, i, cols, 0.0f, b);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (first + r >= rows) continue;
                float f[PER];
                v[r][i].get(f);
#pragma unroll
                for (int j = 0; j < PER; ++j) f[j] = (f[j] - mu[r]) * rs[r] * g[j] + b[j];
                v[r][i].set(f);
                part.store(v[r][i], y + (first + r) * ldy, i, cols);
            }
        }
    }
}

// Rows beyond a block's registers: the row is read in each pass (from L2 after the first).
template <typename T>
__global__ void __launch_bounds__(kLnMostThreads)
    k_layer_norm_fwd_long(const T* __restrict__ x, int64_t ldx, int x_vec, const void* __restrict__ gamma,
                          const void* __restrict__ beta, int w_type, int64_t rows, int cols, float eps,
                          T* __restrict__ y, int64_t ldy, int y_vec, float* __restrict__ mean,
                          float* __restrict__ rstd)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int PER = Vec<T>::kPer;
    __shared__ float red[2][32];
    const float inv = 1.0f / (float)cols;
    const int stride = blockDim.x * PER;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* xr = x + r * ldx;
        Vec<T> v;
        float f[PER], mu[1] = {0.0f}, rs[1] = {0.0f};
        for (int c = threadIdx.x * PER; c < cols; c += stride) {
            v.load(xr, c, cols, x_vec);
            v.get(f);
#pragma unroll
            for (int j = 0; j < PER; ++j) mu[0] += f[j];
        }
        row_sums<1>(mu, blockDim.x, red[0]);
        mu[0] *= inv;
        for (int c = threadIdx.x * PER; c < cols; c += stride) {
            v.load(xr, c, cols, x_vec);
            v.get(f);
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const float d = c + j < cols ? f[j] - mu[0] : 0.0f;
                rs[0] += d * d;
            }
        }
        row_sums<1>(rs, blockDim.x, red[1]);
        rs[0] = 1.0f / sqrtf(rs[0] * inv + eps);
        if (threadIdx.x == 0) {
            if (mean) mean[r] = mu[0];
            if (rstd) rstd[r] = rs[0];
        }
        for (int c = threadIdx.x * PER; c < cols; c += stride) {
            float g[PER], b[PER];
            load_weights<false>(gamma, w_type, c, cols, 1.0f, g);
            load_weights<false>(beta, w_type, c, cols, 0.0f, b);
            v.load(xr, c, cols, x_vec);
            v.get(f);
#pragma unroll
            for (int j = 0; j < PER; ++j) f[j] = (f[j] - mu[0]) * rs[0] * g[j] + b[j];
            v.set(f);
            v.store(y + r * ldy, c, cols, y_vec);
        }
    }
}

// dx, and each block's share of dgamma and dbeta (part: [shares][2][cols], may be null),
// which k_layer_norm_wgrad adds in a fixed order.
template <typename T, int VPT, int R, bool FULL>
__global__ void __launch_bounds__(ln_bwd_threads(VPT))
    k_layer_norm_bwd(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x, int64_t ldx,
                     const void* __restrict__ gamma, int w_type, const float* __restrict__ mean,
                     const float* __restrict__ rstd, int64_t rows, int cols, int tpr, T* __restrict__ dx,
                     int64_t lddx, float* __restrict__ part)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int PER = Vec<T>::kPer;
    __shared__ float red[2][2 * R * 32];
    const int at = threadIdx.x % tpr, group = threadIdx.x / tpr, groups = blockDim.x / tpr;
    const LnColumns<FULL, PER> mine{tpr, at};
    const float inv = 1.0f / (float)cols;
    float g[VPT][PER], sg[VPT][PER], sb[VPT][PER];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        mine.weights(gamma, w_type, i, cols, 1.0f, g[i]);
#pragma unroll
        for (int j = 0; j < PER; ++j) sg[i][j] = sb[i][j] = 0.0f;
    }
    const int64_t step = (int64_t)gridDim.x * groups * R;
    int bank = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * groups * R; r0 < rows; r0 += step, bank ^= 1) {
        const int64_t first = r0 + (int64_t)group * R;
        Vec<T> vd[R][VPT], vx[R][VPT];
        float mu[R], rs[R], s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = first + r < rows;
            mu[r] = in ? mean[first + r] : 0.0f;
            rs[r] = in ? rstd[first + r] : 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (in && mine.first(i) < cols) {
                    mine.load(vd[r][i], dy + (first + r) * lddy, i, cols);
                    mine.load(vx[r][i], x + (first + r) * ldx, i, cols);
                } else {
                    vd[r][i].raw = vx[r][i].raw = make_uint4(0u, 0u, 0u, 0u);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[2 * r] = s[2 * r + 1] = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float d[PER], h[PER];
                vd[r][i].get(d);
                vx[r][i].get(h);
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    // beyond the row's end dy is 0, and with it every term
                    const float hh = (h[j] - mu[r]) * rs[r], dh = d[j] * hh;
                    sg[i][j] += dh;
                    sb[i][j] += d[j];
                    s[2 * r] += d[j] * g[i][j];
                    s[2 * r + 1] += dh * g[i][j];
                }
            }
        }
        if (!dx) continue;
        row_sums<2 * R>(s, tpr, red[bank]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (first + r >= rows) continue;
            const float sa = s[2 * r] * inv, sh = s[2 * r + 1] * inv;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (mine.first(i) >= cols) continue;
                float d[PER], h[PER];
                vd[r][i].get(d);
                vx[r][i].get(h);
#pragma unroll
                for (int j = 0; j < PER; ++j) d[j] = rs[r] * (d[j] * g[i][j] - sa - (h[j] - mu[r]) * rs[r] * sh);
                vd[r][i].set(d);
                mine.store(vd[r][i], dx + (first + r) * lddx, i, cols);
            }
        }
    }
    if (!part) return;
    float* pg = part + (int64_t)blockIdx.x * 2 * cols;
    if (groups > 1) {
        // the block's rows side by side: lanes of a warp by shuffles, the warps one after another
        __shared__ float sum[2][64 * PER];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < PER; ++j)
                for (int o = tpr; o < 32; o *= 2) {
                    sg[i][j] += __shfl_xor_sync(0xffffffffu, sg[i][j], o);
                    sb[i][j] += __shfl_xor_sync(0xffffffffu, sb[i][j], o);
                }
        for (int w = 0; w < (int)blockDim.x / 32; ++w) {
            if ((int)threadIdx.x / 32 == w && (int)(threadIdx.x & 31) < tpr)
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const int c = mine.column(i, j);
                        if (c >= cols) continue;
                        sum[0][c] = w ? sum[0][c] + sg[i][j] : sg[i][j];
                        sum[1][c] = w ? sum[1][c] + sb[i][j] : sb[i][j];
                    }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * cols; c += blockDim.x) pg[c] = c < cols ? sum[0][c] : sum[1][c - cols];
        return;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int c = mine.column(i, j);
            if (c < cols) {
                pg[c] = sg[i][j];
                pg[cols + c] = sb[i][j];
            }
        }
}

// Longer rows: dx in two passes over the row.
template <typename T>
__global__ void __launch_bounds__(kLnMostThreads)
    k_layer_norm_dx_long(const T* __restrict__ dy, int64_t lddy, int dy_vec, const T* __restrict__ x, int64_t ldx,
                         int x_vec, const void* __restrict__ gamma, int w_type, const float* __restrict__ mean,
                         const float* __restrict__ rstd, int64_t rows, int cols, T* __restrict__ dx, int64_t lddx,
                         int dx_vec)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int PER = Vec<T>::kPer;
    __shared__ float red[2][2 * 32];
    const float inv = 1.0f / (float)cols;
    int bank = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, bank ^= 1) {
        const float mu = mean[r], rs = rstd[r];
        float s[2] = {0.0f, 0.0f};
        for (int pass = 0; pass < 2; ++pass) {
            for (int c = threadIdx.x * PER; c < cols; c += blockDim.x * PER) {
                Vec<T> vd, vx;
                float d[PER], h[PER], g[PER];
                vd.load(dy + r * lddy, c, cols, dy_vec);
                vx.load(x + r * ldx, c, cols, x_vec);
                vd.get(d);
                vx.get(h);
                load_weights<false>(gamma, w_type, c, cols, 1.0f, g);
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const float hh = (h[j] - mu) * rs, a = d[j] * g[j];
                    if (pass == 0) {
                        s[0] += a;
                        s[1] += a * hh;
                    } else {
                        d[j] = rs * (a - s[0] - hh * s[1]);
                    }
                }
                if (pass == 1) {
                    vd.set(d);
                    vd.store(dx + r * lddx, c, cols, dx_vec);
                }
            }
            if (pass == 0) {
                row_sums<2>(s, blockDim.x, red[bank]);
                s[0] *= inv;
                s[1] *= inv;
            }
        }
    }
}

// Longer rows: shares of dgamma and dbeta, a block for 256 columns of the rows blockIdx.y, + gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(256)
    k_layer_norm_shares_long(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x, int64_t ldx,
                             const float* __restrict__ mean, const float* __restrict__ rstd, int64_t rows, int cols,
                             float* __restrict__ part)
{
    griddep_wait();
    griddep_launch_dependents();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= cols) return;
    float sg = 0.0f, sb = 0.0f;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const float d = to_f32(dy[r * lddy + c]);
        sg += d * ((to_f32(x[r * ldx + c]) - mean[r]) * rstd[r]);
        sb += d;
    }
    part[(int64_t)blockIdx.y * 2 * cols + c] = sg;
    part[((int64_t)blockIdx.y * 2 + 1) * cols + c] = sb;
}

// ------------------------------------------------------------- a ring of rows
//
// Many long FULL rows: a block walks over groups of R rows that the copy engine brings into a
// ring of stages in shared memory, so that the loads in flight (about 100 KB a block) do not
// depend on registers or on how far the block is in its sums. A stage is free once every
// thread has its part in registers, which the barrier of the row's sums tells. Per element two
// conversions and five or six packed operations remain; with one element to an instruction
// (26 of them) the forward pass took 45 us at 8192 x 4096 bf16, bound by issue.
//
// A wait that runs out (mbar_wait) leaves a wrong result and ITO_ERR_TIMEOUT: later waits return at
// once, every thread still passes every barrier, and the one that asks for copies asks for no more
// and leaves when those under way have landed.
struct LnRing {
    int stages;
    uint32_t row_bytes;
};

// After the last group: the thread that asked for copies gave up at the group `lost`, with a ring's
// worth from that one on under way (as far as there were groups).
__device__ __forceinline__ void ln_unwind(const LnRing& ring, uint64_t* full, int64_t lost, int64_t groups)
{
    const int64_t turn = (lost - blockIdx.x) / gridDim.x, left = (groups - 1 - lost) / gridDim.x + 1;
    ring_landed(full, ring.stages, RingPlace{(int)(turn % ring.stages), (uint32_t)(turn / ring.stages & 1)},
                (int)min((int64_t)ring.stages, left));
}

// Blocks of up to 256 threads: three to an SM forward (8192 x 4096 bf16: 25.6 us, 28.6 with four),
// two backward (43 us, 51 with three, whose registers spill).
constexpr int kLnTight = 3;
constexpr int ln_ring_threads(int vpt, bool tight) { return tight ? 256 : vpt == 4 ? 1024 : 512; }

template <int N>
__device__ __forceinline__ float2 pair_of(const float (&v)[N], int i) { return make_float2(v[2 * i], v[2 * i + 1]); }

// TIGHT: blocks of up to 256 threads, three to an SM
template <typename T, int VPT, int R, bool TIGHT>
__global__ void __launch_bounds__(ln_ring_threads(VPT, TIGHT), TIGHT ? kLnTight : 1)
    k_layer_norm_fwd_ring(const T* __restrict__ x, int64_t ldx, const void* __restrict__ gamma,
                          const void* __restrict__ beta, int w_type, int64_t rows, int cols, float eps,
                          T* __restrict__ y, int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd,
                          LnRing ring, int* __restrict__ err)
{
    static_assert(R <= 2, "rows' roots are taken by every other lane");
    constexpr int PER = Vec<T>::kPer;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[2][R * 32];
    __shared__ uint64_t full[16];
    __shared__ int abort_flag;
    __shared__ int64_t lost;
    const int at = threadIdx.x, tpr = blockDim.x;
    if (at == 0) {
        for (int s = 0; s < ring.stages; ++s) mbar_init(&full[s], 1);
        abort_flag = 0;
        lost = -1;
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const int64_t groups = (rows + R - 1) / R;
    auto fill = [&](int64_t g, int s) {
        if (g >= groups) return;
        const int n = (int)min((int64_t)R, rows - g * R);
        mbar_arrive_expect_tx(&full[s], n * ring.row_bytes);
        for (int r = 0; r < n; ++r)
            bulk_load(smem + (s * R + r) * ring.row_bytes, x + (g * R + r) * ldx, ring.row_bytes, &full[s]);
    };
    if (at == 0)
        for (int s = 0; s < ring.stages; ++s) fill(blockIdx.x + (int64_t)s * gridDim.x, s);
    // a thread's columns stay the same: gamma and beta are registers, where there are enough
    constexpr bool KEEP = VPT <= 2;
    float g[KEEP ? VPT : 1][PER], b[KEEP ? VPT : 1][PER];
    if (KEEP)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            load_weights<true>(gamma, w_type, (i * tpr + at) * PER, cols, 1.0f, g[KEEP ? i : 0]);
            load_weights<true>(beta, w_type, (i * tpr + at) * PER, cols, 0.0f, b[KEEP ? i : 0]);
        }
    const float inv = 1.0f / (float)cols;
    int stage = 0;
    uint32_t phase = 0;
    for (int64_t grp = blockIdx.x; grp < groups; grp += gridDim.x) {
        if (!mbar_wait(&full[stage], phase, &abort_flag, err) && at == 0 && lost < 0) lost = grp;
        float f[R][VPT][PER], mu[R], rs[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (i * tpr + at) * PER;
                Vec<T> v;
                v.raw = make_uint4(0u, 0u, 0u, 0u);
                if (c < cols)
                    v.raw = *reinterpret_cast<const uint4*>(smem + (stage * R + r) * ring.row_bytes + c * sizeof(T));
                v.get(f[r][i]);
#pragma unroll
                for (int j = 0; j < PER / 2; ++j) s = __fadd2_rn(s, pair_of(f[r][i], j));
            }
            mu[r] = s.x + s.y;
        }
        row_sums<R>(mu, tpr, red[0]);
        if (at == 0 && lost < 0) fill(grp + (int64_t)ring.stages * gridDim.x, stage);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mu[r] *= inv;
            float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if ((i * tpr + at) * PER >= cols) continue;
#pragma unroll
                for (int j = 0; j < PER / 2; ++j) {
                    const float2 d = __fadd2_rn(pair_of(f[r][i], j), make_float2(-mu[r], -mu[r]));
                    s = __ffma2_rn(d, d, s);
                    f[r][i][2 * j] = d.x;
                    f[r][i][2 * j + 1] = d.y;
                }
            }
            rs[r] = s.x + s.y;
        }
        row_sums<R>(rs, tpr, red[1]);
        if constexpr (R == 2) {
            // one root and quotient a lane, each row's in every other one
            const float q = 1.0f / sqrtf((threadIdx.x & 1 ? rs[R - 1] : rs[0]) * inv + eps);
            rs[0] = __shfl_sync(0xffffffffu, q, 0);
            rs[R - 1] = __shfl_sync(0xffffffffu, q, 1);
        } else {
            rs[0] = 1.0f / sqrtf(rs[0] * inv + eps);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = grp * R + r;
            if (row >= rows) continue;
            if (at == 0) {
                if (mean) mean[row] = mu[r];
                if (rstd) rstd[row] = rs[r];
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (i * tpr + at) * PER;
                if (c >= cols) continue;
                if (!KEEP) {
                    load_weights<true>(gamma, w_type, c, cols, 1.0f, g[0]);
                    load_weights<true>(beta, w_type, c, cols, 0.0f, b[0]);
                }
#pragma unroll
                for (int j = 0; j < PER / 2; ++j) {
                    const float2 h = __fmul2_rn(pair_of(f[r][i], j), make_float2(rs[r], rs[r]));
                    const float2 o = __ffma2_rn(h, pair_of(g[KEEP ? i : 0], j), pair_of(b[KEEP ? i : 0], j));
                    f[r][i][2 * j] = o.x;
                    f[r][i][2 * j + 1] = o.y;
                }
                Vec<T> v;
                v.set(f[r][i]);
                *reinterpret_cast<uint4*>(y + row * ldy + c) = v.raw;
            }
        }
        if (++stage == ring.stages) { stage = 0; phase ^= 1; }
    }
    if (at == 0 && lost >= 0) ln_unwind(ring, full, lost, groups);
}

template <typename T, int VPT, int R>
__global__ void __launch_bounds__(512)
    k_layer_norm_bwd_ring(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x, int64_t ldx,
                          const void* __restrict__ gamma, int w_type, const float* __restrict__ mean,
                          const float* __restrict__ rstd, int64_t rows, int cols, T* __restrict__ dx, int64_t lddx,
                          float* __restrict__ part, LnRing ring, int* __restrict__ err)
{
    constexpr int PER = Vec<T>::kPer;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[2][2 * R * 32];
    __shared__ uint64_t full[16];
    __shared__ int abort_flag;
    __shared__ int64_t lost;
    const int at = threadIdx.x, tpr = blockDim.x;
    if (at == 0) {
        for (int s = 0; s < ring.stages; ++s) mbar_init(&full[s], 1);
        abort_flag = 0;
        lost = -1;
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const int64_t groups = (rows + R - 1) / R;
    // a stage: R rows of dy, then R rows of x
    auto fill = [&](int64_t g, int s) {
        if (g >= groups) return;
        const int n = (int)min((int64_t)R, rows - g * R);
        mbar_arrive_expect_tx(&full[s], 2 * n * ring.row_bytes);
        for (int r = 0; r < n; ++r) {
            bulk_load(smem + (2 * s * R + r) * ring.row_bytes, dy + (g * R + r) * lddy, ring.row_bytes, &full[s]);
            bulk_load(smem + ((2 * s + 1) * R + r) * ring.row_bytes, x + (g * R + r) * ldx, ring.row_bytes, &full[s]);
        }
    };
    if (at == 0)
        for (int s = 0; s < ring.stages; ++s) fill(blockIdx.x + (int64_t)s * gridDim.x, s);
    constexpr bool KEEP = VPT <= 2;
    float g[KEEP ? VPT : 1][PER];
    float2 sg[VPT][PER / 2], sb[VPT][PER / 2];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (KEEP) load_weights<true>(gamma, w_type, (i * tpr + at) * PER, cols, 1.0f, g[KEEP ? i : 0]);
#pragma unroll
        for (int j = 0; j < PER / 2; ++j) sg[i][j] = sb[i][j] = make_float2(0.0f, 0.0f);
    }
    const float inv = 1.0f / (float)cols;
    int stage = 0, bank = 0;
    uint32_t phase = 0;
    for (int64_t grp = blockIdx.x; grp < groups; grp += gridDim.x, bank ^= 1) {
        float mu[R], rs[R], s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = grp * R + r < rows;
            mu[r] = in ? mean[grp * R + r] : 0.0f;
            rs[r] = in ? rstd[grp * R + r] : 0.0f;
        }
        if (!mbar_wait(&full[stage], phase, &abort_flag, err) && at == 0 && lost < 0) lost = grp;
        Vec<T> vd[R][VPT], vx[R][VPT];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = grp * R + r < rows;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (i * tpr + at) * PER;
                vd[r][i].raw = vx[r][i].raw = make_uint4(0u, 0u, 0u, 0u);
                if (in && c < cols) {
                    vd[r][i].raw =
                        *reinterpret_cast<const uint4*>(smem + (2 * stage * R + r) * ring.row_bytes + c * sizeof(T));
                    vx[r][i].raw = *reinterpret_cast<const uint4*>(smem + ((2 * stage + 1) * R + r) * ring.row_bytes +
                                                                  c * sizeof(T));
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 sa = make_float2(0.0f, 0.0f), sh = make_float2(0.0f, 0.0f);
            const float2 rs2 = make_float2(rs[r], rs[r]), mu2 = make_float2(-mu[r], -mu[r]);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float d[PER], h[PER];
                vd[r][i].get(d);
                vx[r][i].get(h);
                if (!KEEP) load_weights<true>(gamma, w_type, (i * tpr + at) * PER, cols, 1.0f, g[0]);
#pragma unroll
                for (int j = 0; j < PER / 2; ++j) {
                    // beyond the rows' and the row's end dy is 0, and with it every term
                    const float2 dd = pair_of(d, j);
                    const float2 hh = __fmul2_rn(__fadd2_rn(pair_of(h, j), mu2), rs2);
                    const float2 dh = __fmul2_rn(dd, hh);
                    sg[i][j] = __fadd2_rn(sg[i][j], dh);
                    sb[i][j] = __fadd2_rn(sb[i][j], dd);
                    sa = __ffma2_rn(dd, pair_of(g[KEEP ? i : 0], j), sa);
                    sh = __ffma2_rn(dh, pair_of(g[KEEP ? i : 0], j), sh);
                }
            }
            s[2 * r] = sa.x + sa.y;
            s[2 * r + 1] = sh.x + sh.y;
        }
        row_sums<2 * R>(s, tpr, red[bank]);
        if (at == 0 && lost < 0) fill(grp + (int64_t)ring.stages * gridDim.x, stage);
        if (++stage == ring.stages) { stage = 0; phase ^= 1; }
        if (!dx) continue;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = grp * R + r;
            if (row >= rows) continue;
            const float2 rs2 = make_float2(rs[r], rs[r]), mu2 = make_float2(-mu[r], -mu[r]);
            const float2 sa = make_float2(-s[2 * r] * inv, -s[2 * r] * inv);
            const float2 sh = make_float2(-s[2 * r + 1] * inv, -s[2 * r + 1] * inv);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (i * tpr + at) * PER;
                if (c >= cols) continue;
                float d[PER], h[PER];
                vd[r][i].get(d);
                vx[r][i].get(h);
                if (!KEEP) load_weights<true>(gamma, w_type, (i * tpr + at) * PER, cols, 1.0f, g[0]);
#pragma unroll
                for (int j = 0; j < PER / 2; ++j) {
                    const float2 hh = __fmul2_rn(__fadd2_rn(pair_of(h, j), mu2), rs2);
                    const float2 o = __fmul2_rn(__ffma2_rn(hh, sh, __ffma2_rn(pair_of(d, j), pair_of(g[KEEP ? i : 0], j), sa)), rs2);
                    d[2 * j] = o.x;
                    d[2 * j + 1] = o.y;
                }
                vd[r][i].set(d);
                *reinterpret_cast<uint4*>(dx + row * lddx + c) = vd[r][i].raw;
            }
        }
    }
    if (at == 0 && lost >= 0) ln_unwind(ring, full, lost, groups);
    if (!part) return;
    float* pg = part + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < PER / 2; ++j) {
            const int c = (i * tpr + at) * PER + 2 * j;
            if (c < cols) {
                *reinterpret_cast<float2*>(pg + c) = sg[i][j];
                *reinterpret_cast<float2*>(pg + cols + c) = sb[i][j];
            }
        }
}

// The shares' sums: a lane takes a column, a block's warps every 32nd share. (With eight warps
// 304 shares of 4096 columns took as long, 456 of 64 columns 8 us more.)
__global__ void __launch_bounds__(1024)
    k_layer_norm_wgrad(const float* __restrict__ part, int parts, int cols, float* __restrict__ dgamma,
                       float* __restrict__ dbeta)
{
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float sums[32][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < 2 * cols) {
#pragma unroll 4
        for (int p = warp; p < parts; p += 32) s += part[(int64_t)p * 2 * cols + c];
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp || c >= 2 * cols) return;
#pragma unroll
    for (int w = 1; w < 32; ++w) s += sums[w][lane];
    if (c < cols) {
        if (dgamma) dgamma[c] = s;
    } else if (dbeta) {
        dbeta[c - cols] = s;
    }
}

// ------------------------------------------------------------------------ host

// How rows of `cols` elements are shared out among threads.
struct LnShape {
    int vpt;          // vectors a thread holds (0: the row does not fit a block)
    int tpr, block;   // threads of a row and of a block
};

static LnShape ln_shape(int cols, int size, int most)
{
    const int per = 16 / size, vectors = (cols + per - 1) / per;
    LnShape s;
    if (vectors <= 64) {
        // part of a warp, or a warp with two vectors a lane
        s.vpt = vectors <= 32 ? 1 : 2;
        s.tpr = 1;
        while (s.tpr * s.vpt < vectors) s.tpr *= 2;
        s.block = kLnBlock;
        return s;
    }
    // a block: two vectors a thread from 128 threads on, four from 512
    s.vpt = vectors <= 128 ? 1 : vectors <= 1024 ? 2 : 4;
    s.tpr = ((vectors + s.vpt - 1) / s.vpt + 31) / 32 * 32;
    s.block = s.tpr;
    if (s.tpr > most) s = LnShape{0, kLnMostThreads, kLnMostThreads};
    return s;
}

// The ring takes long FULL rows in numbers.
constexpr int kLnRingBytes = 200 * 1024;     // of an SM's blocks together
constexpr int kLnRingRows = 4;               // rows for each SM from which the ring pays

static bool ln_ring_rows(const LnShape& s, int cols, int size, int64_t rows)
{
    return s.vpt && s.tpr > 32 && cols % (16 / size) == 0 && rows >= (int64_t)kLnRingRows * num_sms();
}

// Blocks of an SM: as many threads as the kernel's registers allow, whatever the rows' length
// (20000 x 768 bf16: 15.5 us forward and 26 backward, 30 and 36 with three and two blocks; 8192 x
// 1024 10 and 17, 13.5 and 19; forward 3000 x 10000 35, 59 with one block; 5000 x 2500 f32 18, 27).
static int ln_ring_blocks(const LnShape& s, bool forward)
{
    const int threads = !forward ? 512 : s.vpt == 4 ? 1024 : s.block > 256 ? 640 : kLnTight * 256;   // by their registers
    return std::max(1, threads / s.block);
}

static LnRing ln_ring(const LnShape& s, int cols, int size, int stage_rows, int blocks)
{
    LnRing r;
    r.row_bytes = (uint32_t)cols * size;
    r.stages = std::max(2, std::min(16, kLnRingBytes / blocks / (int)(r.row_bytes * stage_rows)));
    return r;
}

template <typename K>
static int ln_ring_smem(K kern, int bytes)
{
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return set_error(ITO_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(cudaGetLastError()));
    return ITO_OK;
}

// Blocks of the backward pass, and the shares of dgamma and dbeta they leave.
static int ln_bwd_rows(const LnShape& s) { return s.vpt == 1 ? 4 : s.vpt == 2 ? 2 : 1; }

static int ln_bwd_grid(const LnShape& s, int64_t rows)
{
    if (!s.vpt) return (int)std::min<int64_t>(rows, num_sms());
    const int64_t per = (int64_t)(s.block / s.tpr) * ln_bwd_rows(s);
    const int64_t want = (rows + per - 1) / per, most = (int64_t)num_sms() * std::max(1, 768 / s.block);
    return (int)std::min(want, most);
}

static int ln_parts(int64_t rows, int cols, int size)
{
    const LnShape s = ln_shape(cols, size, ln_bwd_threads(4));
    if (!s.vpt) return (int)std::min<int64_t>(rows, 32);
    return ln_bwd_grid(s, rows);
}

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
static int run_fwd(const void* xp, int64_t ldx, const void* gamma, const void* beta, int w_type, int64_t rows,
                   int cols, float eps, void* yp, int64_t ldy, float* mean, float* rstd, cudaStream_t s)
{
    const LnShape sh = ln_shape(cols, sizeof(T), kLnMostThreads);
    const T* x = static_cast<const T*>(xp);
    T* y = static_cast<T*>(yp);
    const int xv = rows_vec(x, ldx, sizeof(T), rows), yv = rows_vec(y, ldy, sizeof(T), rows);
    const int64_t most = (int64_t)num_sms() * (2048 / sh.block);
    if (!sh.vpt) {
        launch_pdl(k_layer_norm_fwd_long<T>, (unsigned)std::min(rows, most), sh.block, 0, s, x, ldx, xv, gamma, beta,
                   w_type, rows, cols, eps, y, ldy, yv, mean, rstd);
        return launch_status("layer norm");
    }
    // several rows at a time once every SM has its blocks of them
    const int groups = sh.block / sh.tpr;
    const int R = sh.vpt <= 2 && rows > (int64_t)4 * groups * num_sms() ? 4 / sh.vpt : 1;
    const int64_t want = (rows + (int64_t)groups * R - 1) / ((int64_t)groups * R);
    const unsigned grid = (unsigned)std::min(want, most);
    const bool full = cols % Vec<T>::kPer == 0 && xv && yv && aligned_to(gamma, 16) && aligned_to(beta, 16);
    if (full && ln_ring_rows(sh, cols, sizeof(T), rows)) {
        const int RR = sh.vpt <= 2 ? 2 : 1;
        const int each = ln_ring_blocks(sh, true);
        const LnRing ring = ln_ring(sh, cols, sizeof(T), RR, each);
        const int smem = ring.stages * RR * (int)ring.row_bytes;
        const unsigned blocks = (unsigned)std::min<int64_t>((rows + RR - 1) / RR, (int64_t)num_sms() * each);
        int* err = device_error_word();
        if (!err) return set_error(ITO_ERR_CUDA, "device error word unavailable");
#define ITO_LN_RING(V, RN, TIGHT)                                                                               \
    do {                                                                                                        \
        const int st = ln_ring_smem(k_layer_norm_fwd_ring<T, V, RN, TIGHT>, smem);                              \
        if (st) return st;                                                                                      \
        launch_pdl(k_layer_norm_fwd_ring<T, V, RN, TIGHT>, blocks, sh.block, smem, s, x, ldx, gamma, beta, w_type, \
                   rows, cols, eps, y, ldy, mean, rstd, ring, err);                                             \
    } while (0)
        if (sh.vpt == 1) ITO_LN_RING(1, 2, true);
        else if (sh.vpt == 2 && sh.block <= 256) ITO_LN_RING(2, 2, true);
        else if (sh.vpt == 2) ITO_LN_RING(2, 2, false);
        else ITO_LN_RING(4, 1, false);
#undef ITO_LN_RING
        return launch_status("layer norm");
    }
#define ITO_LN_AS(V, RR, F)                                                                                       \
    launch_pdl(k_layer_norm_fwd<T, V, RR, F>, grid, sh.block, 0, s, x, ldx, gamma, beta, w_type, rows, cols, \
               sh.tpr, eps, y, ldy, mean, rstd)
#define ITO_LN(V, RR) do { if (full) ITO_LN_AS(V, RR, true); else ITO_LN_AS(V, RR, false); } while (0)
    if (sh.vpt == 1) { if (R > 1) ITO_LN(1, 4); else ITO_LN(1, 1); }
    else if (sh.vpt == 2) { if (R > 1) ITO_LN(2, 2); else ITO_LN(2, 1); }
    else ITO_LN(4, 1);
#undef ITO_LN
#undef ITO_LN_AS
    return launch_status("layer norm");
}

template <typename T>
static int run_bwd(const void* dyp, int64_t lddy, const void* xp, int64_t ldx, const void* gamma, int w_type,
                   const float* mean, const float* rstd, int64_t rows, int cols, float* part, void* dxp, int64_t lddx,
                   float* dgamma, float* dbeta, cudaStream_t s)
{
    const LnShape sh = ln_shape(cols, sizeof(T), ln_bwd_threads(4));
    const T *dy = static_cast<const T*>(dyp), *x = static_cast<const T*>(xp);
    T* dx = static_cast<T*>(dxp);
    const int dyv = rows_vec(dy, lddy, sizeof(T), rows), xv = rows_vec(x, ldx, sizeof(T), rows);
    const int dxv = rows_vec(dx, lddx, sizeof(T), rows);
    const bool wgrad = dgamma || dbeta;
    float* share = wgrad ? part : nullptr;
    const int grid = ln_bwd_grid(sh, rows);
    const bool full = cols % Vec<T>::kPer == 0 && dyv && xv && dxv && aligned_to(gamma, 16);
#define ITO_LN_AS(V, RR, F)                                                                                         \
    launch_pdl(k_layer_norm_bwd<T, V, RR, F>, grid, sh.block, 0, s, dy, lddy, x, ldx, gamma, w_type, mean, \
               rstd, rows, cols, sh.tpr, dx, lddx, share)
#define ITO_LN(V, RR) do { if (full) ITO_LN_AS(V, RR, true); else ITO_LN_AS(V, RR, false); } while (0)
#define ITO_LN_RING(V, RN)                                                                                          \
    do {                                                                                                            \
        const LnRing ring = ln_ring(sh, cols, sizeof(T), 2 * RN, ln_ring_blocks(sh, false));                                                   \
        const int smem = ring.stages * 2 * RN * (int)ring.row_bytes;                                                \
        const int st = ln_ring_smem(k_layer_norm_bwd_ring<T, V, RN>, smem);                                         \
        if (st) return st;                                                                                          \
        parts = (int)std::min<int64_t>((rows + RN - 1) / RN, std::min(parts, num_sms() * ln_ring_blocks(sh, false)));      \
        launch_pdl(k_layer_norm_bwd_ring<T, V, RN>, parts, sh.block, smem, s, dy, lddy, x, ldx, gamma, w_type, mean, \
                   rstd, rows, cols, dx, lddx, share, ring, err);                                                   \
    } while (0)
    int parts = ln_parts(rows, cols, sizeof(T));
    if (full && ln_ring_rows(sh, cols, sizeof(T), rows)) {
        int* err = device_error_word();
        if (!err) return set_error(ITO_ERR_CUDA, "device error word unavailable");
        if (sh.vpt == 1) ITO_LN_RING(1, 2);
        else if (sh.vpt == 2) ITO_LN_RING(2, 2);
        else ITO_LN_RING(4, 1);
    } else if (sh.vpt == 1) ITO_LN(1, 4);
    else if (sh.vpt == 2) ITO_LN(2, 2);
    else if (sh.vpt == 4) ITO_LN(4, 1);
    else {
        // The shares read dy, so they come first where dx replaces it; else dx, after whose two passes the
        // shares find more of both tensors in L2 (3000 x 10000 float32: 195 us, 208 with the shares first).
        const auto shares = [&] {
            if (wgrad)
                launch_pdl(k_layer_norm_shares_long<T>, dim3((cols + 255) / 256, parts), 256, 0, s, dy, lddy, x, ldx,
                           mean, rstd, rows, cols, share);
        };
        if (dx == dy) shares();
        if (dx)
            launch_pdl(k_layer_norm_dx_long<T>, grid, sh.block, 0, s, dy, lddy, dyv, x, ldx, xv, gamma, w_type, mean,
                       rstd, rows, cols, dx, lddx, dxv);
        if (dx != dy) shares();
    }
#undef ITO_LN
#undef ITO_LN_AS
#undef ITO_LN_RING
    if (wgrad)
        launch_pdl(k_layer_norm_wgrad, (2 * cols + 31) / 32, 1024, 0, s, static_cast<const float*>(part),
                   parts, cols, dgamma, dbeta);
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
    // the shares of either element size
    return (size_t)std::max(ln_parts(rows, cols, 2), ln_parts(rows, cols, 4)) * 2 * cols * sizeof(float);
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
