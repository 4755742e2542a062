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
// a warp adds up the rows of a chunk of sorted places, column strip by column strip, and writes each
// token's sum where the token changes. A token whose places go on beyond its chunk leaves pieces, which
// a third kernel joins: a frequent token's thousands of rows are the work of many warps. While one
// cluster of blocks sorts (in the order of 10 us, by latency), the rest of the device writes the zeros of
// the tokens that do not occur.
#include <algorithm>

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
    __device__ __forceinline__ void load_apart(const T* row, int c, int step, int n)
    {
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
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i].store_apart(row, c + i * Vec<T>::kPer * step, step, n);
    }
};

// Lanes that share a row's strip of 8 lanes elements. VEC: lane l holds elements 8 l .. 8 l + 7 of
// the strip (rows on 16-byte boundaries, d a multiple of 8); otherwise l, l + lanes, ..: consecutive
// lanes touch consecutive elements either way.
template <bool VEC, typename T>
__device__ __forceinline__ void load_strip(Eight<T>& e, const T* row, int strip, int lane, int lanes, int d)
{
    if (VEC) e.load(row, strip * 8 * lanes + lane * 8, d);
    else e.load_apart(row, strip * 8 * lanes + lane, lanes, d);
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_strip(const Eight<T>& e, T* row, int strip, int lane, int lanes, int d)
{
    if (VEC) e.store(row, strip * 8 * lanes + lane * 8, d);
    else e.store_apart(row, strip * 8 * lanes + lane, lanes, d);
}

// lanes of a group: as many as a row has vectors, a power of two up to 32
static int row_lanes(int d)
{
    int n = 1;
    while (n < 32 && n * 8 < d) n *= 2;
    return n;
}

// -------------------------------------------------------------------- lookup

constexpr int kEmbThreads = 256;
constexpr int kEmbUnits = 4;         // strips of a group whose loads are in flight together

template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(kEmbThreads)
    k_emb_fwd(const int32_t* __restrict__ ids, int64_t n, const T* __restrict__ table, int64_t ldt, int classes, int d,
              int lanes, int strips, float scale, O* __restrict__ y, int64_t ldy, int* err)
{
    griddep_wait();
    griddep_launch_dependents();
    const int groups = kEmbThreads / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    const int64_t units = n * strips;
    const int64_t first = (int64_t)blockIdx.x * groups * kEmbUnits;
    // (one long division a block; what is left fits 32 bits)
    const int64_t row0 = first / strips;
    const unsigned rest = (unsigned)(first - row0 * strips);
    Eight<T> e[kEmbUnits];
    int id[kEmbUnits];
#pragma unroll
    for (int u = 0; u < kEmbUnits; ++u) {
        const unsigned at = rest + u * groups + group;
        const int64_t row = row0 + at / (unsigned)strips;
        id[u] = first + u * groups + group < units ? ids[row] : -1;
    }
#pragma unroll
    for (int u = 0; u < kEmbUnits; ++u) {
        const unsigned at = rest + u * groups + group;
        const int strip = (int)(at % (unsigned)strips);
        const bool in = id[u] >= 0 && id[u] < classes;
        if (!in && id[u] != -1 && strip == 0 && lane == 0) raise_device_error(err, ITO_ERR_ARG);
        load_strip<VEC>(e[u], table + (in ? id[u] * ldt : 0), strip, lane, lanes, in ? d : 0);
    }
#pragma unroll
    for (int u = 0; u < kEmbUnits; ++u) {
        if (first + u * groups + group >= units) break;
        const unsigned at = rest + u * groups + group;
        const int64_t row = row0 + at / (unsigned)strips;
        float f[8];
        e[u].get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= scale;
        Eight<O> o;
        o.set(f);
        store_strip<VEC>(o, y + row * ldy, (int)(at % (unsigned)strips), lane, lanes, d);
    }
}

// ------------------------------------------------------- sorting places by token

// A stable sort by digits of 8 bits, lowest first, by one cluster of blocks: each warp counts the
// digits of its own run of places, the counts of a block's warps and of the cluster's blocks are
// summed up to where each warp's places of each digit go, and the warps write them there. Runs are
// consecutive, so places of equal digits keep their order. A place without a token has the key
// `classes`, behind all others.
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kSortCluster = 8;
constexpr int kZeroRows = 16384;     // rows of the table whose presence a block notes at a time

struct EmbSort {
    const int32_t* ids;
    int n, classes, passes, blocks;  // blocks that sort
    int32_t* keys[2];                // [n] each: the last pass writes keys[0], places[0]
    int32_t* places[2];
    void* table;                     // rows of absent tokens get zeros (null: they stay)
    int64_t row_bytes, pitch_bytes;
    int wide;                        // 16-byte stores
    int* err;
};

__device__ __forceinline__ void emb_sort(const EmbSort& a)
{
    __shared__ unsigned counts[kSortWarps][256];
    __shared__ unsigned total[256], base[256], scan[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, block = (int)cluster_ctarank();
    const int per = (a.n + a.blocks * kSortWarps - 1) / (a.blocks * kSortWarps);     // places of a warp
    const int64_t lo = (int64_t)(block * kSortWarps + warp) * per;
    const int64_t hi = min((int64_t)a.n, lo + per);
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = 8 * pass, to = (a.passes - 1 - pass) & 1;
        auto key_at = [&](int64_t i) -> int {
            if (pass) return __ldcg(a.keys[to ^ 1] + i);
            const int id = a.ids[i];
            return id >= 0 && id < a.classes ? id : a.classes;
        };
        for (int i = threadIdx.x; i < kSortWarps * 256; i += kSortThreads) (&counts[0][0])[i] = 0;
        __syncthreads();
        for (int64_t i = lo; i < hi; i += 32) {
            const bool in = i + lane < hi;
            const int key = in ? key_at(i + lane) : 0;
            const unsigned digit = in ? (unsigned)key >> shift & 255 : 256;
            const unsigned same = __match_any_sync(0xffffffffu, digit);
            if (in && lane == __ffs(same) - 1) counts[warp][digit] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        if (threadIdx.x < 256) {
            unsigned sum = 0;
            for (int w = 0; w < kSortWarps; ++w) {
                const unsigned c = counts[w][threadIdx.x];
                counts[w][threadIdx.x] = sum;
                sum += c;
            }
            total[threadIdx.x] = sum;
        }
        cluster_sync();
        if (threadIdx.x < 256) {
            unsigned before = 0, all = 0;
            for (int b = 0; b < a.blocks; ++b) {
                unsigned c;
                asm volatile("ld.shared::cluster.u32 %0, [%1];"
                             : "=r"(c)
                             : "r"(mapa_shared(smem_u32(&total[threadIdx.x]), b))
                             : "memory");
                if (b < block) before += c;
                all += c;
            }
            unsigned inc = all;              // inclusive sums over the digits
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned c = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += c;
            }
            if (lane == 31) scan[warp] = inc;
            base[threadIdx.x] = before + inc - all;
        }
        __syncthreads();
        if (threadIdx.x < 256) {
            unsigned lower = 0;
            for (int w = 0; w < warp; ++w) lower += scan[w];
            base[threadIdx.x] += lower;
        }
        __syncthreads();
        for (int64_t i = lo; i < hi; i += 32) {
            const bool in = i + lane < hi;
            const int key = in ? key_at(i + lane) : 0;
            const int place = !in ? 0 : pass ? __ldcg(a.places[to ^ 1] + i + lane) : (int)(i + lane);
            const unsigned digit = in ? (unsigned)key >> shift & 255 : 256;
            const unsigned same = __match_any_sync(0xffffffffu, digit);
            if (in) {
                const unsigned at = base[digit] + counts[warp][digit] + __popc(same & ((1u << lane) - 1));
                a.keys[to][at] = key;
                a.places[to][at] = place;
            }
            __syncwarp();
            if (in && lane == __ffs(same) - 1) counts[warp][digit] += __popc(same);
            __syncwarp();
        }
        cluster_sync();                      // the pass is written, and the blocks' totals are read
    }
}

// zeros for the rows of tokens that do not occur, block `b` of `blocks`
__device__ __forceinline__ void emb_zero(const EmbSort& a, int b, int blocks)
{
    __shared__ unsigned there[kZeroRows / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (a.classes + blocks - 1) / blocks;
    const int64_t end = min((int64_t)a.classes, (int64_t)(b + 1) * per);
    for (int64_t r0 = (int64_t)b * per; r0 < end; r0 += kZeroRows) {
        const int rows = (int)min((int64_t)kZeroRows, end - r0);
        __syncthreads();
        for (int i = threadIdx.x; i < (rows + 31) / 32; i += kSortThreads) there[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < a.n; i += kSortThreads) {
            const int64_t r = a.ids[i] - r0;
            if (r >= 0 && r < rows) atomicOr(&there[r >> 5], 1u << (r & 31));
        }
        __syncthreads();
        for (int r = warp; r < rows; r += kSortWarps) {
            if (there[r >> 5] >> (r & 31) & 1) continue;
            char* row = static_cast<char*>(a.table) + (r0 + r) * a.pitch_bytes;
            if (a.wide) {
                for (int64_t i = lane * 16; i < a.row_bytes; i += 512)
                    *reinterpret_cast<uint4*>(row + i) = make_uint4(0u, 0u, 0u, 0u);
            } else {
                for (int64_t i = lane * 2; i < a.row_bytes; i += 64) *reinterpret_cast<uint16_t*>(row + i) = 0;
            }
        }
    }
}

__global__ void __launch_bounds__(kSortThreads) k_emb_sort(const __grid_constant__ EmbSort a)
{
    griddep_wait();
    griddep_launch_dependents();
    if ((int)blockIdx.x < a.blocks) {
        for (int i = blockIdx.x * kSortThreads + threadIdx.x; i < a.n; i += a.blocks * kSortThreads) {
            const int id = a.ids[i];
            if (id < -1 || id >= a.classes) raise_device_error(a.err, ITO_ERR_ARG);
        }
        emb_sort(a);
    } else {
        emb_zero(a, (int)blockIdx.x - a.blocks, (int)gridDim.x - a.blocks);
    }
}

// ----------------------------------------------------------- sums of sorted places

// A warp's chunk of sorted places holds runs of equal tokens. A run that began before the chunk leaves
// its sum in head[chunk]; one that begins in the chunk and goes on behind it in tail[chunk]; others
// are whole and go to the table.
constexpr int kSumThreads = 256;
constexpr int kSumAhead = 4;         // rows of dy whose loads are in flight together

struct EmbSum {
    const int32_t *keys, *places;
    int n, classes, d, chunk, chunks, strips;
    const void* dy;
    int64_t lddy;
    float scale;
    int add;
    void* table;
    int64_t ldt;
    float *head, *tail;              // [chunks][pitch]
    int pitch;
};

template <typename O, bool VEC>
__device__ __forceinline__ void emb_put(const EmbSum& a, int key, int strip, int lane, const float (&s)[8])
{
    O* row = static_cast<O*>(a.table) + (int64_t)key * a.ldt;
    Eight<O> o;
    float f[8];
    if (a.add) {
        load_strip<VEC>(o, static_cast<const O*>(row), strip, lane, 32, a.d);
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

template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(kSumThreads) k_emb_sum(const __grid_constant__ EmbSum a)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t unit = (int64_t)blockIdx.x * (kSumThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (unit >= (int64_t)a.chunks * a.strips) return;
    const int chunk = (int)(unit / a.strips), strip = (int)(unit % a.strips);
    const int lo = chunk * a.chunk, len = min(a.chunk, a.n - lo);
    // (a chunk has 32 places at most: one to a lane)
    const int mine = lane < len ? __ldg(a.keys + lo + lane) : a.classes;
    const int place = lane < len ? __ldg(a.places + lo + lane) : 0;
    int before = -1, after = -1;
    if (lo > 0) before = __ldg(a.keys + lo - 1);
    if (lo + len < a.n) after = __ldg(a.keys + lo + len);
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
    bool from_before = before == __shfl_sync(0xffffffffu, mine, 0);
    const int64_t at = (int64_t)chunk * a.pitch + strip * 256 + lane * 8;
    for (int i0 = 0; i0 < len; i0 += kSumAhead) {
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
            if (key >= a.classes) return;            // places without a token are the last
            float f[8];
            e[u].get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] += f[j];
            const int next = i + 1 < len ? __shfl_sync(0xffffffffu, mine, i + 1 & 31) : after;
            if (next == key && i + 1 < len) continue;
            if (from_before) piece_store(a.head + at, s);
            else if (next == key) piece_store(a.tail + at, s);
            else emb_put<O, VEC>(a, key, strip, lane, s);
            from_before = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = 0.0f;
        }
    }
}

// A block to a chunk's strip: where a token's run begins in the chunk and goes on, its pieces are
// added, a share of the chunks that it goes on through to each warp, and the shares in their order.
template <typename O, bool VEC>
__global__ void __launch_bounds__(kSumThreads) k_emb_join(const __grid_constant__ EmbSum a)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int WARPS = kSumThreads / 32;
    __shared__ float part[WARPS][256];
    const int chunk = (int)(blockIdx.x / a.strips), strip = (int)(blockIdx.x % a.strips);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int end = (chunk + 1) * a.chunk;           // the chunk's last place is end - 1; (end <= n - 1 here)
    const int key = __ldg(a.keys + end - 1);
    if (key >= a.classes || __ldg(a.keys + end) != key) return;
    if (chunk > 0 && __ldg(a.keys + chunk * a.chunk) == key && __ldg(a.keys + chunk * a.chunk - 1) == key) return;
    // the run's end: the first place from `end` on with another key, 32 guesses at a time
    int lo = end, hi = a.n;                          // keys[lo] == key; the end is in lo + 1 .. hi
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int64_t guess = lo + (int64_t)step * (lane + 1);
        const unsigned same = __ballot_sync(0xffffffffu, guess < hi && __ldg(a.keys + guess) == key);
        const int got = __popc(same);                // (the keys are sorted: a prefix of the guesses)
        const int64_t up = lo + (int64_t)step * (got + 1);
        lo += step * got;
        hi = (int)min((int64_t)hi, up);
    }
    const int last = (hi - 1) / a.chunk;             // the chunk that the run ends in
    const int more = last - chunk, per = (more + WARPS - 1) / WARPS;
    const int64_t at = strip * 256 + lane * 8;
    const int c0 = chunk + 1 + warp * per, c1 = min(last + 1, c0 + per);
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
    if (warp == 0) {
        const float4* p = reinterpret_cast<const float4*>(a.tail + (int64_t)chunk * a.pitch + at);
        const float4 x = p[0], y = p[1];
        s[0] = x.x; s[1] = x.y; s[2] = x.z; s[3] = x.w;
        s[4] = y.x; s[5] = y.y; s[6] = y.z; s[7] = y.w;
    }
#pragma unroll 4
    for (int c = c0; c < c1; ++c) {
        const float4* p = reinterpret_cast<const float4*>(a.head + (int64_t)c * a.pitch + at);
        const float4 x = p[0], y = p[1];
        s[0] += x.x; s[1] += x.y; s[2] += x.z; s[3] += x.w;
        s[4] += y.x; s[5] += y.y; s[6] += y.z; s[7] += y.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[warp][lane * 8 + i] = s[i];
    __syncthreads();
    if (warp) return;
    for (int w = 1; w < WARPS; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += part[w][lane * 8 + i];
    emb_put<O, VEC>(a, key, strip, lane, s);
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
    const int lanes = row_lanes(d), strips = (d + 8 * lanes - 1) / (8 * lanes);
    const int64_t per = (int64_t)kEmbThreads / lanes * kEmbUnits, blocks = (n * strips + per - 1) / per;
    if (blocks > INT32_MAX) return set_error(ITO_ERR_SHAPE, "too many elements");
    launch_pdl(vec ? k_emb_fwd<T, O, true> : k_emb_fwd<T, O, false>, (unsigned)blocks, kEmbThreads, 0, s, ids, n,
               static_cast<const T*>(table), ldt, classes, d, lanes, strips, scale, static_cast<O*>(y), ldy, err);
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

// Places of a chunk: 32, or 8 where 32 would leave SMs without a warp's work.
static int sum_chunk(int64_t n, int strips) { return n / 32 * strips >= 8 * kNumSMsHint ? 32 : 8; }

struct EmbLayout {
    int strips, chunk, chunks, pitch;
    size_t keys, pieces, bytes;      // of one array of keys or places; of heads or tails; of all
};

static EmbLayout emb_layout(int64_t n, int d)
{
    EmbLayout l;
    l.strips = (d + 255) / 256;
    l.chunk = sum_chunk(n, l.strips);
    l.chunks = (int)((n + l.chunk - 1) / l.chunk);
    l.pitch = l.strips * 256;
    l.keys = align256((size_t)n * 4);
    l.pieces = align256((size_t)l.chunks * l.pitch * 4);
    l.bytes = 4 * l.keys + 2 * l.pieces;
    return l;
}

template <typename T, typename O>
static int run_emb_sum(const EmbSum& a, bool vec, cudaStream_t s)
{
    const int64_t units = (int64_t)a.chunks * a.strips, blocks = (units + kSumThreads / 32 - 1) / (kSumThreads / 32);
    launch_pdl(vec ? k_emb_sum<T, O, true> : k_emb_sum<T, O, false>, (unsigned)blocks, kSumThreads, 0, s, a);
    if (a.chunks > 1)
        launch_pdl(vec ? k_emb_join<O, true> : k_emb_join<O, false>, (unsigned)((int64_t)(a.chunks - 1) * a.strips),
                   kSumThreads, 0, s, a);
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
    if (type == ITO_F32) return run_emb_fwd_to<float>(out_type, ids, n, table, ldt, classes, d, vec, scale, y, ldy, err, s);
    if (type == ITO_BF16)
        return run_emb_fwd_to<__nv_bfloat16>(out_type, ids, n, table, ldt, classes, d, vec, scale, y, ldy, err, s);
    return run_emb_fwd_to<__half>(out_type, ids, n, table, ldt, classes, d, vec, scale, y, ldy, err, s);
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
    if ((int64_t)l.chunks * l.strips > INT32_MAX) return set_error(ITO_ERR_SHAPE, "too many elements");
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
    // 2048 places a block and more: fewer take the cluster's barriers longer than the places
    for (q.blocks = 1; q.blocks < kSortCluster && q.blocks * 2048 < n; q.blocks *= 2) {}
    for (int i = 0; i < 2; ++i) {
        q.keys[i] = reinterpret_cast<int32_t*>(ws + i * l.keys);
        q.places[i] = reinterpret_cast<int32_t*>(ws + (2 + i) * l.keys);
    }
    q.table = add ? nullptr : dtable;
    q.row_bytes = (int64_t)d * type_bytes(out_type);
    q.pitch_bytes = ldt * (int64_t)type_bytes(out_type);
    q.wide = aligned_to(dtable, 16) && q.row_bytes % 16 == 0 && (classes == 1 || q.pitch_bytes % 16 == 0);
    q.err = err;
    // zeros: a block to an SM beside the sorting cluster, and no more than there are rows
    int zero = 0;
    if (!add) zero = (std::min(2 * num_sms(), classes) + q.blocks - 1) / q.blocks * q.blocks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(q.blocks + zero));
    cfg.blockDim = dim3(kSortThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = q.blocks;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_emb_sort, q);
    if (e != cudaSuccess) return set_error(ITO_ERR_CUDA, "embedding backward launch: %s", cudaGetErrorString(e));

    EmbSum a{};
    a.keys = q.keys[0];
    a.places = q.places[0];
    a.n = (int)n;
    a.classes = classes;
    a.d = d;
    a.chunk = l.chunk;
    a.chunks = l.chunks;
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
    const bool vec = rows_in_eights(dy, type, lddy, n, d) && rows_in_eights(dtable, out_type, ldt, classes, d);
    if (type == ITO_F32) return run_emb_sum<float, float>(a, vec, s);
    if (type == ITO_BF16)
        return out_type == ITO_F32 ? run_emb_sum<__nv_bfloat16, float>(a, vec, s)
                                   : run_emb_sum<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
    return out_type == ITO_F32 ? run_emb_sum<__half, float>(a, vec, s) : run_emb_sum<__half, __half>(a, vec, s);
}

}  // extern "C"
