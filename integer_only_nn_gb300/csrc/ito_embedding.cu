// Embedding lookup with its scale, and the table's gradient by sorted tokens.
//
//   y_i = scale table[id_i]        dtable[v] = scale sum of dy_i over the places i with id_i = v
//
// An id of -1 stands for no token: its y is 0, its dy takes no part.
//
// The lookup is a copy: a group of lanes to a row (as many as the row has vectors of 8 elements, up
// to a warp), so that narrow rows share warps. Its floor is the table's rows read and y written.
//
// The gradient sums rows of dy that are far apart. Places are sorted by token first (stably, so the
// order of every sum is the places' own and equal calls give equal bits; no atomics on the sums), then
// warps add up the rows of chunks of sorted places, a strip of columns each, and write a token's sum where
// the token changes. A token whose places go on into the next chunk leaves pieces, which are joined in
// the block, and over blocks by a third kernel: a frequent token's thousands of rows are the work of many warps. The rows of
// tokens that do not occur get zeros while pieces are joined, which leaves most of the device idle (some of
// them while the places are sorted: 47 us instead of 41 for 34586 x 304 of 15292, 126 instead of 123 for
// 16384 x 4096 of 32768, because the presence of a token is then not known from the sorted ones).
#include <algorithm>
#include <climits>
#include <cmath>

#include "ito_float.cuh"

namespace ito {

// eight consecutive elements of a row, as 32-bit floats, or eight that are `step` apart; those from
// n on are 0 (loads) or left alone (stores)
template <typename T>
struct Eight {
    static constexpr int kVecs = 8 / Vec<T>::kPer;
    Vec<T> v[kVecs];

    __device__ __forceinline__ void load(const T* row, int c, int n) // (c + 8 <= n or c >= n, aligned)
    {
        if (c < n) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i].raw = *reinterpret_cast<const uint4*>(row + c + i * Vec<T>::kPer);
        } else {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i].raw = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    // KEPT: nothing is written there while the kernel runs
    template <bool KEPT>
    __device__ __forceinline__ void load_apart(const T* row, int c, int step, int n)
    {
        if (c + 7 * step < n) {              // all of them: no look at each
            const T* p = row + c;
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i, p += step) {
                using Bits = typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type;
                const Bits* q = reinterpret_cast<const Bits*>(p);
                w[i] = KEPT ? __ldg(q) : *q;
            }
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < kVecs; ++i) v[i].raw = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            } else {
                v[0].raw = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i].load_apart(row, c + i * Vec<T>::kPer * step, step, n);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            float p[Vec<T>::kPer];
            v[i].get(p);
#pragma unroll
            for (int j = 0; j < Vec<T>::kPer; ++j) f[i * Vec<T>::kPer + j] = p[j];
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            float p[Vec<T>::kPer];
#pragma unroll
            for (int j = 0; j < Vec<T>::kPer; ++j) p[j] = f[i * Vec<T>::kPer + j];
            v[i].set(p);
        }
    }
    __device__ __forceinline__ void store(T* row, int c, int n) const
    {
        if (c >= n) return;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) *reinterpret_cast<uint4*>(row + c + i * Vec<T>::kPer) = v[i].raw;
    }
    __device__ __forceinline__ void store_apart(T* row, int c, int step, int n) const
    {
        if (c + 7 * step < n) {
            T* p = row + c;
#pragma unroll
            for (int i = 0; i < 8; ++i, p += step) {
                const uint4 r = v[i / Vec<T>::kPer].raw;
                const uint32_t w[4] = {r.x, r.y, r.z, r.w};
                if constexpr (sizeof(T) == 4) *reinterpret_cast<uint32_t*>(p) = w[i & 3];
                else *reinterpret_cast<uint16_t*>(p) = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i].store_apart(row, c + i * Vec<T>::kPer * step, step, n);
    }
};

// Lanes that share a row's strip of 8 lanes elements. VEC: lane l holds elements 8 l .. 8 l + 7 of
// the strip (rows on 16-byte boundaries, d a multiple of 8); otherwise l, l + lanes, ..: consecutive
// lanes touch consecutive elements either way.
template <bool VEC, bool KEPT = true, typename T>
__device__ __forceinline__ void load_strip(Eight<T>& e, const T* row, int strip, int lane, int lanes, int d)
{
    if (VEC) e.load(row, strip * 8 * lanes + lane * 8, d);
    else e.template load_apart<KEPT>(row, strip * 8 * lanes + lane, lanes, d);
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_strip(const Eight<T>& e, T* row, int strip, int lane, int lanes, int d)
{
    if (VEC) e.store(row, strip * 8 * lanes + lane * 8, d);
    else e.store_apart(row, strip * 8 * lanes + lane, lanes, d);
}

// lanes of a group: as many as a row has vectors, a power of two up to 32; -> its logarithm
static int row_lanes(int d)
{
    int n = 0;
    while (n < 5 && 8 << n < d) ++n;
    return n;
}

// -------------------------------------------------------------------- lookup

constexpr int kEmbThreads = 256;
constexpr int kEmbUnits = 4;         // strips of a group whose loads are in flight together

template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(kEmbThreads)
    k_emb_fwd(const int32_t* __restrict__ ids, int64_t n, const T* __restrict__ table, int64_t ldt, int classes, int d,
              int log_lanes, Divider strips, float scale, O* __restrict__ y, int64_t ldy, int* err)
{
    griddep_wait();
    griddep_launch_dependents();
    const int lanes = 1 << log_lanes, groups = kEmbThreads >> log_lanes, group = threadIdx.x >> log_lanes;
    const int lane = threadIdx.x & (lanes - 1);
    const int64_t first = (int64_t)blockIdx.x * groups * kEmbUnits;
    // (one long division a block; what is left fits 32 bits)
    const int64_t row0 = first / strips.d;
    const unsigned rest = (unsigned)(first - row0 * strips.d);
    const unsigned units = (unsigned)min((int64_t)groups * kEmbUnits, n * strips.d - first);
    unsigned row[kEmbUnits];
    int id[kEmbUnits];
#pragma unroll
    for (int u = 0; u < kEmbUnits; ++u) {
        const unsigned k = u * groups + group;
        row[u] = strips(rest + k);
        id[u] = k < units ? __ldg(ids + row0 + row[u]) : -1;
    }
    Eight<T> e[kEmbUnits];
#pragma unroll
    for (int u = 0; u < kEmbUnits; ++u) {
        const int strip = (int)(rest + u * groups + group - row[u] * strips.d);
        const bool in = (unsigned)id[u] < (unsigned)classes;
        if (!in && id[u] != -1 && strip == 0 && lane == 0) raise_device_error(err, ITO_ERR_ARG);
        load_strip<VEC>(e[u], table + (in ? id[u] * ldt : 0), strip, lane, lanes, in ? d : 0);
    }
    O* const out = y + row0 * ldy;
#pragma unroll
    for (int u = 0; u < kEmbUnits; ++u) {
        const unsigned k = u * groups + group;
        if (k >= units) break;
        Eight<O> o;
        if (std::is_same<T, O>::value && scale == 1.0f) {
            o = reinterpret_cast<const Eight<O>&>(e[u]);
        } else {
            float f[8];
            e[u].get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= scale;
            o.set(f);
        }
        store_strip<VEC>(o, out + row[u] * ldy, (int)(rest + k - row[u] * strips.d), lane, lanes, d);
    }
}

// 16-bit rows at any alignment, of the table and of y: a thread writes the eight elements of y in one aligned
// 16 bytes, which begin anywhere in the table's row (Eight16); one by one at a row's two ends. `eights`
// aligned eights touch a row at most. (30000 x 1001 of 32768 rows: 24 us; elements one by one 38.)
constexpr int kEmbShifted = 2;       // eights of a thread whose loads are in flight together

template <typename T, typename O>
__global__ void __launch_bounds__(kEmbThreads, 5)
    k_emb_fwd_shifted(const int32_t* __restrict__ ids, int64_t n, const T* __restrict__ table, int64_t ldt, int classes,
                      int d, Divider eights, float scale, O* __restrict__ y, int64_t ldy, int* err)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int PER = kEmbThreads * kEmbShifted;
    const uint16_t* const lo = reinterpret_cast<const uint16_t*>(table);
    const uint16_t* const hi = lo + (classes - 1) * ldt + d;
    const int64_t first = (int64_t)blockIdx.x * PER, total = n * eights.d;
    const int64_t row0 = first / eights.d;
    const unsigned rest = (unsigned)(first - row0 * eights.d), left = (unsigned)min((int64_t)PER, total - first);
    int id[kEmbShifted], col[kEmbShifted];
    uint16_t* to[kEmbShifted];
#pragma unroll
    for (int u = 0; u < kEmbShifted; ++u) {
        const unsigned j = u * kEmbThreads + threadIdx.x, r = eights(rest + j);
        id[u] = j < left ? __ldg(ids + row0 + r) : -1;
        to[u] = reinterpret_cast<uint16_t*>(y) + (row0 + r) * ldy;
        // the row's first aligned eight begins up to seven elements before it
        col[u] = (int)(rest + j - r * eights.d) * 8 - (int)(reinterpret_cast<uintptr_t>(to[u]) >> 1 & 7);
        if (j >= left) col[u] = d;
        if (id[u] >= classes || id[u] < 0) {
            if (id[u] != -1 && col[u] <= 0) raise_device_error(err, ITO_ERR_ARG);
            id[u] = -1;
        }
    }
    Eight16 e[kEmbShifted];
#pragma unroll
    for (int u = 0; u < kEmbShifted; ++u) {
#pragma unroll
        for (int i = 0; i < 5; ++i) e[u].w[i] = 0u;
        if (id[u] < 0) continue;
        const uint16_t* row = lo + id[u] * ldt;
        if (col[u] >= 0 && col[u] + 8 <= d && Eight16::whole(row + col[u], lo, hi)) {
            e[u].load(row + col[u]);
        } else {                                     // as `load` leaves them for these eight
            uint16_t x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = col[u] + i >= 0 && col[u] + i < d ? __ldg(row + col[u] + i) : 0;
            const bool half = reinterpret_cast<uintptr_t>(row + col[u]) & 2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e[u].w[i] = half ? (uint32_t)x[2 * i] << 16 | (i ? x[2 * i - 1] : 0) : x[2 * i] | (uint32_t)x[2 * i + 1] << 16;
            }
            e[u].w[4] = half ? x[7] : 0;
        }
    }
#pragma unroll
    for (int u = 0; u < kEmbShifted; ++u) {
        if (col[u] >= d) continue;
        Vec<T> v;
        v.raw = e[u].get(lo + (id[u] < 0 ? 0 : id[u] * ldt) + col[u]);
        Vec<O> o;
        if (std::is_same<T, O>::value && scale == 1.0f) {
            o.raw = v.raw;
        } else {
            float f[8];
            v.get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= scale;
            o.set(f);
        }
        if (col[u] >= 0 && col[u] + 8 <= d) {
            *reinterpret_cast<uint4*>(to[u] + col[u]) = o.raw;
        } else {
            const uint32_t w[4] = {o.raw.x, o.raw.y, o.raw.z, o.raw.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col[u] + i >= 0 && col[u] + i < d) to[u][col[u] + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// a row of zeros by a warp: 16 bytes at a time, its ends up to the next 16-byte boundary by elements of 2
__device__ __forceinline__ void zero_row(char* row, int64_t bytes, int lane)
{
    char* const end = row + bytes;
    char* const a = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(row) + 15) & ~uintptr_t(15));
    char* const b = reinterpret_cast<char*>(reinterpret_cast<uintptr_t>(end) & ~uintptr_t(15));
    for (char* p = a + lane * 16; p < b; p += 512) *reinterpret_cast<uint4*>(p) = make_uint4(0u, 0u, 0u, 0u);
    char* const head = a < b ? a : end;              // (a row may lie within 32 bytes)
    if (row + lane * 2 < head) *reinterpret_cast<uint16_t*>(row + lane * 2) = 0;
    if (a < b && b + lane * 2 < end) *reinterpret_cast<uint16_t*>(b + lane * 2) = 0;
}

// The rows of places without a token, a warp to a place, after a lookup with a scale that is not finite: the
// lookup's kernels multiply their zeros by it. (Looked at there, the lookup takes 43.2 us instead of 40.5 for 16384 x 4096
// bf16 and 37 instead of 31 for 30000 x 1001 from float32.)
__global__ void __launch_bounds__(kEmbThreads)
    k_emb_none(const int32_t* __restrict__ ids, int64_t n, int classes, void* y, int64_t pitch_bytes, int64_t row_bytes)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t warps = (int64_t)gridDim.x * (kEmbThreads / 32);
    for (int64_t i = (int64_t)blockIdx.x * (kEmbThreads / 32) + (threadIdx.x >> 5); i < n; i += warps)
        if ((unsigned)__ldg(ids + i) >= (unsigned)classes)
            zero_row(static_cast<char*>(y) + i * pitch_bytes, row_bytes, threadIdx.x & 31);
}

// ------------------------------------------------------- sorting places by token

// A stable sort by digits of 8 bits, lowest first, by one cluster of 16 blocks or 8: each warp counts the
// digits of its own run of places, the counts of a block's warps and of the cluster's blocks are
// summed up to where each warp's places of each digit go, and the warps write them there. Runs are
// consecutive, so places of equal digits keep their order. A place without a token has the key
// `classes`, behind all others.
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortCluster = 16;
// A few places are sorted by counting, for each, those that go before it: a comparison for each pair, on all
// SMs, without a barrier between blocks (the whole gradient of 2047 x 787, added: 13.4 us, and 15.7 with the
// digits' passes; of 4000: 19.9 and 17.6).
constexpr int kRankMost = 2048, kRankThreads = 256, kRankParts = 8, kRankPlaces = kRankThreads / kRankParts;

struct EmbSort {
    const int32_t* ids;
    int n, classes, passes, blocks;  // blocks that sort
    int32_t* keys[2];                // [n] each: the last pass writes keys[0], places[0]
    int32_t* places[2];
    int* err;
};

struct SortSums {
    unsigned counts[kSortWarps][256];    // of a warp's digits, then where the warp's places of a digit begin
    unsigned quarter[4][256], total[256], base[256], scan[8];
};

// From the warps' counts to where each warp's places of each digit begin: counts becomes the block's
// exclusive sums over its warps, base[digit] the cluster's place of the block's first.
__device__ __forceinline__ void sort_offsets(SortSums& q, int blocks, int block)
{
    const int t = threadIdx.x, d = t & 255, lane = t & 31, warp = t >> 5;
    constexpr int W = kSortWarps / 4;    // four threads to a digit
    const int w0 = (t >> 8) * W;
    unsigned c[W], sum = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) c[w] = q.counts[w0 + w][d];
#pragma unroll
    for (int w = 0; w < W; ++w) sum += c[w];
    q.quarter[t >> 8][d] = sum;
    __syncthreads();
    unsigned first = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) first += i < t >> 8 ? q.quarter[i][d] : 0;
    if (t >> 8 == 3) q.total[d] = first + sum;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        q.counts[w0 + w][d] = first;
        first += c[w];
    }
    cluster_sync();
    if (t < 256) {
        unsigned of[kSortCluster], before = 0, all = 0;
#pragma unroll
        for (int b = 0; b < kSortCluster; ++b) {
            of[b] = 0;
            if (b < blocks)
                asm volatile("ld.shared::cluster.u32 %0, [%1];"
                             : "=r"(of[b])
                             : "r"(mapa_shared(smem_u32(&q.total[t]), b))
                             : "memory");
        }
#pragma unroll
        for (int b = 0; b < kSortCluster; ++b) {
            if (b < block) before += of[b];
            all += of[b];
        }
        unsigned inc = all;              // inclusive sums over the digits
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) q.scan[warp] = inc;
        q.base[t] = before + inc - all;
    }
    __syncthreads();
    if (t < 256) {
        unsigned lower = 0;
        for (int w = 0; w < warp; ++w) lower += q.scan[w];
        q.base[t] += lower;
    }
    __syncthreads();
}

// The lanes whose digit (of 8 bits) is this lane's, by a vote on each bit: a match over the warp in one
// instruction takes longer (34586 places in 8 blocks: 30 us, 34 with it).
__device__ __forceinline__ unsigned same_digit(unsigned digit)
{
    unsigned same = 0xffffffffu;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const bool bit = digit >> b & 1;
        const unsigned with = __ballot_sync(0xffffffffu, bit);
        same &= bit ? with : ~with;
    }
    return same;
}

__device__ __forceinline__ int emb_key(const EmbSort& a, int id) { return id >= 0 && id < a.classes ? id : a.classes; }

// Up to 1024 R places a block: R to a lane, kept in registers between the passes and
// exchanged through the blocks' shared memory. Places beyond n have a key above all and stay the last.
template <int R>
__device__ __forceinline__ void emb_sort_held(const EmbSort& a, SortSums& q, int* exchange)
{
    constexpr int HOLD = R * kSortThreads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, block = (int)cluster_ctarank();
    int* const xkeys = exchange;
    int* const xplaces = exchange + HOLD;
    int key[R], place[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        place[r] = block * HOLD + (warp * R + r) * 32 + lane;
        key[r] = place[r] < a.n ? emb_key(a, __ldg(a.ids + place[r])) : INT_MAX;
    }
    for (int pass = 0; pass < a.passes; ++pass) {
        unsigned rank[R];
        for (int i = lane; i < 256; i += 32) q.counts[warp][i] = 0;
        __syncwarp();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const unsigned digit = (unsigned)key[r] >> (8 * pass) & 255;
            const unsigned same = same_digit(digit);
            const unsigned so_far = q.counts[warp][digit];
            __syncwarp();
            if (lane == __ffs(same) - 1) q.counts[warp][digit] = so_far + __popc(same);
            __syncwarp();
            rank[r] = so_far + __popc(same & ((1u << lane) - 1));
        }
        __syncthreads();
        sort_offsets(q, a.blocks, block);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const unsigned digit = (unsigned)key[r] >> (8 * pass) & 255;
            const int at = (int)(q.base[digit] + q.counts[warp][digit] + rank[r]);
            if (pass + 1 < a.passes) {
                const int to = at / HOLD, i = at % HOLD;
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(xkeys + i), to)), "r"(key[r])
                             : "memory");
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(xplaces + i), to)), "r"(place[r])
                             : "memory");
            } else if (at < a.n) {
                a.keys[0][at] = key[r];
                a.places[0][at] = place[r];
            }
        }
        cluster_sync();                  // the exchange is written, and the blocks' totals are read
        if (pass + 1 < a.passes) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                key[r] = xkeys[(warp * R + r) * 32 + lane];
                place[r] = xplaces[(warp * R + r) * 32 + lane];
            }
        }
    }
}

// Any number of places, which go through memory from pass to pass.
__device__ __forceinline__ void emb_sort(const EmbSort& a, SortSums& q)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, block = (int)cluster_ctarank();
    const int per = (a.n + a.blocks * kSortWarps - 1) / (a.blocks * kSortWarps);     // places of a warp
    const int64_t lo = (int64_t)(block * kSortWarps + warp) * per;
    const int64_t hi = min((int64_t)a.n, lo + per);
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = 8 * pass, to = (a.passes - 1 - pass) & 1;
        auto key_at = [&](int64_t i) -> int { return pass ? __ldcg(a.keys[to ^ 1] + i) : emb_key(a, a.ids[i]); };
        for (int i = lane; i < 256; i += 32) q.counts[warp][i] = 0;
        __syncwarp();
        for (int64_t i = lo; i < hi; i += 32) {
            const bool in = i + lane < hi;
            const int key = in ? key_at(i + lane) : 0;
            const unsigned digit = (unsigned)key >> shift & 255;
            const unsigned same = same_digit(digit) & __ballot_sync(0xffffffffu, in);
            if (in && lane == __ffs(same) - 1) q.counts[warp][digit] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        sort_offsets(q, a.blocks, block);
        for (int64_t i = lo; i < hi; i += 32) {
            const bool in = i + lane < hi;
            const int key = in ? key_at(i + lane) : 0;
            const int place = !in ? 0 : pass ? __ldcg(a.places[to ^ 1] + i + lane) : (int)(i + lane);
            const unsigned digit = (unsigned)key >> shift & 255;
            const unsigned same = same_digit(digit) & __ballot_sync(0xffffffffu, in);
            if (in) {
                const unsigned at = q.base[digit] + q.counts[warp][digit] + __popc(same & ((1u << lane) - 1));
                a.keys[to][at] = key;
                a.places[to][at] = place;
            }
            __syncwarp();
            if (in && lane == __ffs(same) - 1) q.counts[warp][digit] += __popc(same);
            __syncwarp();
        }
        cluster_sync();                      // the pass is written, and the blocks' totals are read
    }
}

__device__ __forceinline__ void check_ids(const EmbSort& a, int first, int step)
{
    for (int i = first; i < a.n; i += step) {
        const int id = a.ids[i];
        if (id < -1 || id >= a.classes) raise_device_error(a.err, ITO_ERR_ARG);
    }
}

// R: places a lane holds (0: they go through memory)
template <int R>
__global__ void __launch_bounds__(kSortThreads) k_emb_sort(const __grid_constant__ EmbSort a)
{
    extern __shared__ int exchange[];
    __shared__ SortSums sums;
    griddep_wait();
    griddep_launch_dependents();
    if constexpr (R > 0) emb_sort_held<R>(a, sums, exchange);
    else emb_sort(a, sums);
    check_ids(a, blockIdx.x * kSortThreads + threadIdx.x, a.blocks * kSortThreads);
}

// Eight threads to a place, each of which compares a share of the keys: those that are smaller, or equal and
// earlier, go before it.
__global__ void __launch_bounds__(kRankThreads) k_emb_rank(const __grid_constant__ EmbSort a)
{
    __shared__ int4 keys[kRankMost / 4];
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x == 0) check_ids(a, threadIdx.x, kRankThreads);
    const int vecs = (a.n + 4 * kRankParts - 1) / (4 * kRankParts) * kRankParts;     // padded with keys above all
    for (int i0 = threadIdx.x; i0 < 4 * vecs; i0 += 8 * kRankThreads) {
        int id[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) id[u] = i0 + u * kRankThreads < a.n ? __ldg(a.ids + i0 + u * kRankThreads) : -1;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + u * kRankThreads, key = id[u] >= 0 && id[u] < a.classes ? id[u] : a.classes;
            if (i < 4 * vecs) reinterpret_cast<int*>(keys)[i] = i < a.n ? key : INT_MAX;
        }
    }
    __syncthreads();
    const int place = blockIdx.x * kRankPlaces + threadIdx.x / kRankParts, part = threadIdx.x % kRankParts;
    const int mine = place < a.n ? reinterpret_cast<const int*>(keys)[place] : 0;
    int before = 0;
#pragma unroll 4
    for (int v = part; v < vecs; v += kRankParts) {
        const int4 k = keys[v];
        // keys of earlier places go before an equal one (those behind it in its own vector are taken out below)
        const int limit = 4 * v < place ? mine + 1 : mine;
        before += (k.x < limit) + (k.y < limit) + (k.z < limit) + (k.w < limit);
    }
    if (place < a.n && place / 4 % kRankParts == part)
        for (int i = place; i < (place | 3) + 1; ++i)
            before -= place % 4 != 0 && reinterpret_cast<const int*>(keys)[i] == mine;
#pragma unroll
    for (int o = 1; o < kRankParts; o <<= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    if (place < a.n && part == 0) {
        a.keys[0][before] = mine;
        a.places[0][before] = place;
    }
}

// ----------------------------------------------------------- sums of sorted places

// A block adds the rows of a span of sorted places, a chunk to each warp. A run of equal tokens that begins
// and ends in a chunk is whole and goes to the table; the pieces of one that goes on into the next chunks
// meet in shared memory, in their order. What began before the span leaves its sum in head[span], what
// goes on behind it in tail[span], for k_emb_join.
constexpr int kSumThreads = 256;
constexpr int kSumWarps = kSumThreads / 32;
constexpr int kSumAhead = 4;         // rows of dy whose loads are in flight together

struct EmbSum {
    const int32_t *keys, *places;
    int n, classes, d, strips;
    int chunk, span, spans;          // places of a warp, of a block; blocks' worth of places
    const void* dy;
    int64_t lddy;
    float scale;
    int add;
    void* table;
    int64_t ldt;
    float *head, *tail;              // [spans][pitch]
    int pitch;
    int join_blocks;                 // the others of the joining kernel write zeros to the rows of absent tokens
    int zero_rows;                   // of a warp
    int64_t row_bytes, pitch_bytes;
};

// The rows of absent tokens, zero_rows to a warp (32 KB, 32 rows at most, 16 warps to an SM at least): each lane looks its row up among
// the sorted keys, and runs of absent rows are zeroed at once where nothing lies between rows. (512 KB to a
// warp: the sums' kernel, which these were part of, took 190 us instead of 100 for 16384 x 4096 and 32768
// tokens, because too few warps were left to keep the memory busy.)
__device__ __forceinline__ void emb_zero_rest(const EmbSum& a, int64_t warp, int lane)
{
    const int64_t r0 = warp * a.zero_rows, row = r0 + lane;
    bool absent = false;
    if (lane < a.zero_rows && row < a.classes) {
        int lo = 0, hi = a.n;                        // the first key that is not below `row` is in lo .. hi
        while (lo < hi) {
            const int mid = lo + (hi - lo) / 2;
            if (__ldg(a.keys + mid) < row) lo = mid + 1;
            else hi = mid;
        }
        absent = lo == a.n || __ldg(a.keys + lo) != row;
    }
    const bool dense = a.pitch_bytes == a.row_bytes;
    for (unsigned rows = __ballot_sync(0xffffffffu, absent); rows;) {
        const int first = __ffs(rows) - 1;
        const unsigned gap = ~(rows >> first);       // its lowest bit: the length of the run of rows
        const int run = dense ? (gap ? __ffs(gap) - 1 : 32) : 1;
        zero_row(static_cast<char*>(a.table) + (r0 + first) * a.pitch_bytes, run * a.row_bytes, lane);
        rows &= run + first >= 32 ? 0u : ~0u << (run + first);
    }
}

template <typename O, bool VEC>
__device__ __forceinline__ void emb_put(const EmbSum& a, int key, int strip, int lane, const float (&s)[8])
{
    O* row = static_cast<O*>(a.table) + (int64_t)key * a.ldt;
    Eight<O> o;
    float f[8];
    if (a.add) {
        load_strip<VEC, false>(o, static_cast<const O*>(row), strip, lane, 32, a.d);
        o.get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += a.scale * s[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = a.scale * s[i];
    }
    o.set(f);
    store_strip<VEC>(o, row, strip, lane, 32, a.d);
}

// a piece's strip in the workspace: lane l's eight at 8 l whatever the rows' layout
__device__ __forceinline__ void piece_store(float* p, const float (&s)[8])
{
    reinterpret_cast<float4*>(p)[0] = make_float4(s[0], s[1], s[2], s[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(s[4], s[5], s[6], s[7]);
}

__device__ __forceinline__ void add_piece(float (&s)[8], const float* p)
{
    const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
    s[0] += x.x; s[1] += x.y; s[2] += x.z; s[3] += x.w;
    s[4] += y.x; s[5] += y.y; s[6] += y.z; s[7] += y.w;
}

template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(kSumThreads) k_emb_sum(const __grid_constant__ EmbSum a)
{
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float heads[kSumWarps][256], tails[kSumWarps][256];
    __shared__ int state[kSumWarps];                 // of a warp's chunk: it has a head, that goes on; it has a tail
    constexpr int HEAD = 1, ON = 2, TAIL = 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int span = (int)(blockIdx.x / a.strips), strip = (int)(blockIdx.x % a.strips);
    const int64_t lo = (int64_t)span * a.span + warp * a.chunk;
    const int len = (int)max((int64_t)0, min((int64_t)a.chunk, a.n - lo));
    // (a chunk has 32 places at most: one to a lane)
    const int mine = lane < len ? __ldg(a.keys + lo + lane) : a.classes;
    const int place = lane < len ? __ldg(a.places + lo + lane) : 0;
    int before = -1, after = -1;
    if (lo > 0 && len) before = __ldg(a.keys + lo - 1);
    if (lo + len < a.n) after = __ldg(a.keys + lo + len);
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
    bool from_before = before == __shfl_sync(0xffffffffu, mine, 0), none = false;
    int st = 0, tail_key = 0;
    for (int i0 = 0; i0 < len && !none; i0 += kSumAhead) {
        Eight<T> e[kSumAhead];
#pragma unroll
        for (int u = 0; u < kSumAhead; ++u) {
            const int i = i0 + u;
            const int key = __shfl_sync(0xffffffffu, mine, i & 31), p = __shfl_sync(0xffffffffu, place, i & 31);
            load_strip<VEC>(e[u], static_cast<const T*>(a.dy) + (int64_t)p * a.lddy, strip, lane, 32,
                            i < len && key < a.classes ? a.d : 0);
        }
#pragma unroll
        for (int u = 0; u < kSumAhead; ++u) {
            const int i = i0 + u;
            if (i >= len) break;
            const int key = __shfl_sync(0xffffffffu, mine, i);
            none = key >= a.classes;                 // places without a token are the last
            if (none) break;
            float f[8];
            e[u].get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] += f[j];
            const int next = i + 1 < len ? __shfl_sync(0xffffffffu, mine, i + 1 & 31) : after;
            if (next == key && i + 1 < len) continue;
            if (from_before) {
                piece_store(&heads[warp][lane * 8], s);
                st |= next == key ? HEAD | ON : HEAD;
            } else if (next == key) {
                piece_store(&tails[warp][lane * 8], s);
                st |= TAIL;
                tail_key = key;
            } else {
                emb_put<O, VEC>(a, key, strip, lane, s);
            }
            from_before = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = 0.0f;
        }
    }
    if (lane == 0) state[warp] = st;
    __syncthreads();
    const int64_t at = (int64_t)span * a.pitch + strip * 256 + lane * 8;
    // a run from this warp's tail on, and (warp 0) the one from before the span
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        if (which ? warp || !(st & HEAD) : !(st & TAIL)) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = 0.0f;
        add_piece(s, which ? &heads[0][lane * 8] : &tails[warp][lane * 8]);
        bool on = which ? st & ON : true;
        for (int w = warp + 1; on && w < kSumWarps; ++w) {
            add_piece(s, &heads[w][lane * 8]);
            on = state[w] & ON;
        }
        if (which) piece_store(a.head + at, s);
        else if (on) piece_store(a.tail + at, s);
        else emb_put<O, VEC>(a, tail_key, strip, lane, s);
    }
}

// A block to eight strips of a span: where a token's run begins in the span and goes on, its pieces are
// added. Of a few pieces each warp adds its strip's; of many (a run through kJoinAlone spans and more)
// every strip's are shared among the warps, and the shares added in their order.
constexpr int kJoinWarps = kSumThreads / 32, kJoinAlone = 64;

template <typename O, bool VEC>
__global__ void __launch_bounds__(kSumThreads) k_emb_join(const __grid_constant__ EmbSum a)
{
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float part[kJoinWarps][256];
    const int groups = (a.strips + kJoinWarps - 1) / kJoinWarps;
    const int span = (int)(blockIdx.x / groups), strip0 = (int)(blockIdx.x % groups) * kJoinWarps;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((int)blockIdx.x >= a.join_blocks) {
        emb_zero_rest(a, (int64_t)(blockIdx.x - a.join_blocks) * kJoinWarps + warp, lane);
        return;
    }
    const int end = (span + 1) * a.span;             // the span's last place is end - 1 (and end < n here)
    const int key = __ldg(a.keys + end - 1), first = __ldg(a.keys + span * a.span);
    const int before = span > 0 ? __ldg(a.keys + span * a.span - 1) : -1;
    if (key >= a.classes || __ldg(a.keys + end) != key) return;
    if (first == key && before == key) return;
    // the span that the run ends in: 32 spans at a time, those at whose ends it goes on (a prefix of them)
    int last = span + 1;
    for (;;) {
        const int64_t next = (int64_t)(last + lane + 1) * a.span;
        const int on = __popc(__ballot_sync(0xffffffffu, next < a.n && __ldg(a.keys + next) == key));
        last += on;
        if (on < 32) break;
    }
    const int more = last - span;
    if (more < kJoinAlone) {
        const int strip = strip0 + warp;
        if (strip >= a.strips) return;
        const int64_t at = strip * 256 + lane * 8;
        float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        add_piece(s, a.tail + (int64_t)span * a.pitch + at);
#pragma unroll 16
        for (int c = span + 1; c <= last; ++c) add_piece(s, a.head + (int64_t)c * a.pitch + at);
        emb_put<O, VEC>(a, key, strip, lane, s);
        return;
    }
    const int per = (more + kJoinWarps - 1) / kJoinWarps;
    const int c0 = span + 1 + warp * per, c1 = min(last + 1, c0 + per);
    for (int strip = strip0; strip < min(a.strips, strip0 + kJoinWarps); ++strip) {
        const int64_t at = strip * 256 + lane * 8;
        float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (warp == 0) add_piece(s, a.tail + (int64_t)span * a.pitch + at);
#pragma unroll 8
        for (int c = c0; c < c1; ++c) add_piece(s, a.head + (int64_t)c * a.pitch + at);
#pragma unroll
        for (int i = 0; i < 8; ++i) part[warp][lane * 8 + i] = s[i];
        __syncthreads();
        if (warp == 0) {
            for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] += part[w][lane * 8 + i];
            emb_put<O, VEC>(a, key, strip, lane, s);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------------ host

static int check_emb(int64_t n, int classes, int d)
{
    if (n < 1 || classes < 1 || d < 1) return set_error(ITO_ERR_SHAPE, "sizes must be >= 1");
    if (n > (1 << 30) || classes > (1 << 30)) return set_error(ITO_ERR_SHAPE, "more than 2^30 tokens or rows");
    if (d > (1 << 24)) return set_error(ITO_ERR_SHAPE, "d above 2^24");
    return ITO_OK;
}

static int check_rows(const void* p, int type, int64_t ld, int64_t rows, int d, const char* name)
{
    if (!p) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    if (!type_known(type)) return set_error(ITO_ERR_ARG, "%s: unknown type", name);
    if (!aligned_to(p, type_bytes(type))) return set_error(ITO_ERR_ARG, "%s: misaligned pointer", name);
    if (rows > 1 && ld < d) return set_error(ITO_ERR_SHAPE, "%s: row stride below its columns", name);
    return ITO_OK;
}

static bool rows_in_eights(const void* p, int type, int64_t ld, int64_t rows, int d)
{
    return d % 8 == 0 && rows_vec(p, ld, type_bytes(type), rows);
}

template <typename T, typename O>
static int run_emb_fwd(const int32_t* ids, int64_t n, const void* table, int64_t ldt, int classes, int d, bool vec,
                       float scale, void* y, int64_t ldy, int* err, cudaStream_t s)
{
    if constexpr (sizeof(T) == 2 && sizeof(O) == 2) {
        if (!vec && d >= 16) {
            const Divider eights(d / 8 + 2);         // (d elements that begin at any of an eight's)
            const int64_t blocks = (n * eights.d + kEmbThreads * kEmbShifted - 1) / (kEmbThreads * kEmbShifted);
            if (blocks > INT32_MAX) return set_error(ITO_ERR_SHAPE, "too many elements");
            launch_pdl(k_emb_fwd_shifted<T, O>, (unsigned)blocks, kEmbThreads, 0, s, ids, n, static_cast<const T*>(table),
                       ldt, classes, d, eights, scale, static_cast<O*>(y), ldy, err);
            return launch_status("embedding");
        }
    }
    const int log_lanes = row_lanes(d), lanes = 1 << log_lanes, strips = (d + 8 * lanes - 1) / (8 * lanes);
    const int64_t per = (int64_t)kEmbThreads / lanes * kEmbUnits, blocks = (n * strips + per - 1) / per;
    if (blocks > INT32_MAX) return set_error(ITO_ERR_SHAPE, "too many elements");
    launch_pdl(vec ? k_emb_fwd<T, O, true> : k_emb_fwd<T, O, false>, (unsigned)blocks, kEmbThreads, 0, s, ids, n,
               static_cast<const T*>(table), ldt, classes, d, log_lanes, Divider(strips), scale, static_cast<O*>(y), ldy, err);
    return launch_status("embedding");
}

template <typename T>
static int run_emb_fwd_to(int out_type, const int32_t* ids, int64_t n, const void* table, int64_t ldt, int classes, int d,
                          bool vec, float scale, void* y, int64_t ldy, int* err, cudaStream_t s)
{
    if (out_type == ITO_F32) return run_emb_fwd<T, float>(ids, n, table, ldt, classes, d, vec, scale, y, ldy, err, s);
    if (out_type == ITO_BF16)
        return run_emb_fwd<T, __nv_bfloat16>(ids, n, table, ldt, classes, d, vec, scale, y, ldy, err, s);
    return run_emb_fwd<T, __half>(ids, n, table, ldt, classes, d, vec, scale, y, ldy, err, s);
}

static size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// Places of a chunk: 32, or fewer down to 4 where that many would leave an SM fewer than 32 warps' work.
static int sum_chunk(int64_t n, int strips)
{
    int chunk = 32;
    while (chunk > 4 && n / chunk * strips < 32 * kNumSMsHint) chunk /= 2;
    return chunk;
}

static void sort_launch(cudaLaunchConfig_t* cfg, cudaLaunchAttribute (&at)[2], int blocks, size_t bytes, cudaStream_t s)
{
    cfg->gridDim = dim3((unsigned)blocks);
    cfg->blockDim = dim3(kSortThreads);
    cfg->dynamicSmemBytes = bytes;
    cfg->stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = blocks;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg->attrs = at;
    cfg->numAttrs = 2;
}

template <int R>
static int run_emb_sort(const EmbSort& q, cudaStream_t s)
{
    constexpr int BYTES = R * kSortThreads * 8;
    static OnEachDevice ready;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess)
        e = ready.run(device, [&] {
            const cudaError_t f = cudaFuncSetAttribute(k_emb_sort<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
            return f == cudaSuccess ? cudaFuncSetAttribute(k_emb_sort<R>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) : f;
        });
    if (e != cudaSuccess) return set_error(ITO_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    sort_launch(&cfg, at, q.blocks, BYTES, s);
    e = cudaLaunchKernelEx(&cfg, k_emb_sort<R>, q);
    return e == cudaSuccess ? ITO_OK : set_error(ITO_ERR_CUDA, "embedding backward launch: %s", cudaGetErrorString(e));
}

// Whether a cluster of 16 blocks that sort fits on this device (8 always do).
static bool sort_in_sixteen()
{
    static std::atomic<int> known{0};                // (the same on each device of this part)
    if (!known) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute at[2];
        sort_launch(&cfg, at, 16, 4 * kSortThreads * 8, nullptr);
        cfg.numAttrs = 1;
        int got = 0;
        const bool fits = cudaFuncSetAttribute(k_emb_sort<4>, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kSortThreads * 8) == cudaSuccess &&
                          cudaFuncSetAttribute(k_emb_sort<4>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                          cudaOccupancyMaxActiveClusters(&got, k_emb_sort<4>, &cfg) == cudaSuccess && got > 0;
        if (!fits) cudaGetLastError();
        known = fits ? 16 : 8;
    }
    return known == 16;
}

struct EmbLayout {
    int strips, chunk, span, spans, pitch;
    size_t keys, pieces, bytes;      // of one array of keys or places; of heads or tails; of all
};

static EmbLayout emb_layout(int64_t n, int d)
{
    EmbLayout l;
    l.strips = (d + 255) / 256;
    l.chunk = sum_chunk(n, l.strips);
    l.span = kSumWarps * l.chunk;
    l.spans = (int)((n + l.span - 1) / l.span);
    l.pitch = l.strips * 256;
    l.keys = align256((size_t)n * 4);
    l.pieces = align256((size_t)l.spans * l.pitch * 4);
    l.bytes = 4 * l.keys + 2 * l.pieces;
    return l;
}

template <typename T, typename O>
static int run_emb_sum(EmbSum a, bool vec, cudaStream_t s)
{
    launch_pdl(vec ? k_emb_sum<T, O, true> : k_emb_sum<T, O, false>, (unsigned)(a.spans * a.strips), kSumThreads, 0, s, a);
    const int groups = (a.strips + kJoinWarps - 1) / kJoinWarps;
    a.zero_rows = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(32, 32768 / a.row_bytes), a.classes / (16 * num_sms())));
    const int zero = a.add ? 0 : (a.classes + a.zero_rows * kJoinWarps - 1) / (a.zero_rows * kJoinWarps);
    a.join_blocks = (a.spans - 1) * groups;
    if (a.join_blocks + zero)
        launch_pdl(vec ? k_emb_join<O, true> : k_emb_join<O, false>, (unsigned)(a.join_blocks + zero), kSumThreads, 0, s, a);
    return launch_status("embedding backward");
}

}  // namespace ito

using namespace ito;

extern "C" {

int ito_embedding_fwd(const int32_t* ids, int64_t n, const void* table, int64_t ldt, int type, int classes, int d,
                      float scale, int out_type, void* y, int64_t ldy, void* stream)
{
    if (!ids) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    if (!aligned_to(ids, 4)) return set_error(ITO_ERR_ARG, "ids: misaligned pointer");
    int r = check_emb(n, classes, d);
    if (!r) r = check_rows(table, type, ldt, classes, d, "table");
    if (!r) r = check_rows(y, out_type, ldy, n, d, "y");
    if (r) return r;
    int* err = device_error_word();
    if (!err) return set_error(ITO_ERR_CUDA, "device error word unavailable");
    const bool vec = rows_in_eights(table, type, ldt, classes, d) && rows_in_eights(y, out_type, ldy, n, d);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (type == ITO_F32) r = run_emb_fwd_to<float>(out_type, ids, n, table, ldt, classes, d, vec, scale, y, ldy, err, s);
    else if (type == ITO_BF16)
        r = run_emb_fwd_to<__nv_bfloat16>(out_type, ids, n, table, ldt, classes, d, vec, scale, y, ldy, err, s);
    else r = run_emb_fwd_to<__half>(out_type, ids, n, table, ldt, classes, d, vec, scale, y, ldy, err, s);
    if (r || std::isfinite(scale)) return r;
    const int64_t size = type_bytes(out_type);
    launch_pdl(k_emb_none, (unsigned)std::min<int64_t>((n + kEmbThreads / 32 - 1) / (kEmbThreads / 32), 8 * num_sms()), kEmbThreads, 0,
               s, ids, n, classes, y, ldy * size, d * size);
    return launch_status("embedding");
}

size_t ito_embedding_bwd_workspace_size(int64_t n, int classes, int d)
{
    return check_emb(n, classes, d) ? 0 : emb_layout(n, d).bytes;
}

int ito_embedding_bwd(const void* dy, int64_t lddy, int type, const int32_t* ids, int64_t n, int classes, int d,
                      float scale, int add, int out_type, void* workspace, size_t workspace_bytes, void* dtable,
                      int64_t ldt, void* stream)
{
    if (!ids) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    if (!aligned_to(ids, 4)) return set_error(ITO_ERR_ARG, "ids: misaligned pointer");
    int r = check_emb(n, classes, d);
    if (!r) r = check_rows(dy, type, lddy, n, d, "dy");
    if (!r) r = check_rows(dtable, out_type, ldt, classes, d, "dtable");
    if (r) return r;
    if (out_type != type && out_type != ITO_F32) return set_error(ITO_ERR_ARG, "out_type must be type or ITO_F32");
    const EmbLayout l = emb_layout(n, d);
    if ((int64_t)l.spans * l.strips > INT32_MAX) return set_error(ITO_ERR_SHAPE, "too many elements");
    if (!workspace) return set_error(ITO_ERR_ARG, "workspace is NULL");
    if (!aligned_to(workspace, 256)) return set_error(ITO_ERR_ARG, "workspace not 256-byte aligned");
    if (workspace_bytes < l.bytes) return set_error(ITO_ERR_ARG, "workspace too small");
    int* err = device_error_word();
    if (!err) return set_error(ITO_ERR_CUDA, "device error word unavailable");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);

    EmbSort q{};
    q.ids = ids;
    q.n = (int)n;
    q.classes = classes;
    for (q.passes = 1; q.passes < 4 && (classes >> (8 * q.passes)); ++q.passes) {}
    for (int i = 0; i < 2; ++i) {
        q.keys[i] = reinterpret_cast<int32_t*>(ws + i * l.keys);
        q.places[i] = reinterpret_cast<int32_t*>(ws + (2 + i) * l.keys);
    }
    const bool rank = n <= kRankMost;
    q.err = err;
    if (rank) {
        q.blocks = (int)((n + kRankPlaces - 1) / kRankPlaces);
        launch_pdl(k_emb_rank, (unsigned)q.blocks, kRankThreads, 0, s, q);
        r = launch_status("embedding backward");
        if (r) return r;
    } else {
        // (34586 places: 20 us in 16 blocks, 29 in 8)
        q.blocks = n > 8192 && sort_in_sixteen() ? 16 : 8;
        const int64_t each = (n + q.blocks * kSortThreads - 1) / (q.blocks * kSortThreads);
        r = each <= 1 ? run_emb_sort<1>(q, s) : each <= 2 ? run_emb_sort<2>(q, s) : each <= 4 ? run_emb_sort<4>(q, s)
            : run_emb_sort<0>(q, s);
        if (r) return r;
    }

    EmbSum a{};
    a.keys = q.keys[0];
    a.places = q.places[0];
    a.n = (int)n;
    a.classes = classes;
    a.d = d;
    a.chunk = l.chunk;
    a.span = l.span;
    a.spans = l.spans;
    a.strips = l.strips;
    a.dy = dy;
    a.lddy = lddy;
    a.scale = scale;
    a.add = add != 0;
    a.table = dtable;
    a.ldt = ldt;
    a.head = reinterpret_cast<float*>(ws + 4 * l.keys);
    a.tail = reinterpret_cast<float*>(ws + 4 * l.keys + l.pieces);
    a.pitch = l.pitch;
    a.row_bytes = (int64_t)d * type_bytes(out_type);
    a.pitch_bytes = ldt * (int64_t)type_bytes(out_type);
    const bool vec = rows_in_eights(dy, type, lddy, n, d) && rows_in_eights(dtable, out_type, ldt, classes, d);
    if (type == ITO_F32) return run_emb_sum<float, float>(a, vec, s);
    if (type == ITO_BF16)
        return out_type == ITO_F32 ? run_emb_sum<__nv_bfloat16, float>(a, vec, s)
                                   : run_emb_sum<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
    return out_type == ITO_F32 ? run_emb_sum<__half, float>(a, vec, s) : run_emb_sum<__half, __half>(a, vec, s);
}

}  // extern "C"
