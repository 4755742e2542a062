// Log probabilities of given tokens (class labels), with the distribution's entropy and its
// largest alternatives, and the gradient of the first two.
//
//   top = max x    s = sum exp(x - top)    lse = top + log s
//   logp = x[target] - lse                 H = log s - (sum (x - top) exp(x - top)) / s
//   dx_j = g_logp (hot_j - p_j) - g_H p_j (log p_j + H),      p = exp(x - lse)
//
// Masked classes hold -inf: they have p = 0 and take no part. A row whose every class is
// masked has lse = -inf, log probabilities of -inf, entropy 0 and a gradient of 0. A target
// of -1 stands for no token: logp 0 and no gradient from it.
#include <algorithm>
#include <climits>
#include <cmath>

#include "ito_float.cuh"

namespace ito {

constexpr int kLpMaxTop = 32;        // alternatives: a warp's list holds one to a lane
constexpr int kLpWarps = 8;          // warps of a block
constexpr int kLpCluster = 8;        // blocks that share a long row, at most
constexpr float kLog2e = 1.4426950408889634f;

// An element as a number that orders alternatives: larger values first, equal ones by their index,
// a NaN above all. 0 is below every element.
typedef unsigned long long Key;

__device__ __forceinline__ uint32_t value_order(float v)
{
    const uint32_t b = v == v ? __float_as_uint(v + 0.0f) : 0x7FFFFFFFu;     // (-0 ties with 0)
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ Key make_key(float v, int i) { return (Key)value_order(v) << 32 | (0xFFFFFFFFu - (uint32_t)i); }
__device__ __forceinline__ float key_value(Key k)
{
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ int key_index(Key k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ---------------------------------------------------------- sums of a part of a row
//
// One pass in powers of two: with L = log2 e and c = top L (rounded), y = x L - c in one rounding,
// s = sum 2^y and t = sum y 2^y, brought to a new `top` when a round of elements raises it
// (rarely, after the first few). c's own rounding cancels in H = ln 2 (log2 s - t / s) and in
// log p = ln 2 (y - log2 s), while it is small beside 1: `top` starts at -2^20, where masked
// elements of -inf add 0 and so do finite ones far below, and a row whose largest element lies
// outside +-2^20 (s stays below 1/2, or top ends above) is taken again by FarSums.
constexpr float kLpReach = 1048576.0f;
constexpr float kLpStart = -kLpReach;
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float max_nan(float a, float b)      // a NaN wins
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct Sums {
    float top, s, t;             // t: of y 2^y, y counted from top

    __device__ __forceinline__ void clear()
    {
        top = kLpStart;
        s = t = 0.0f;
    }
    // To a top no smaller: by the difference of the two c, each rounded as the sums' own was. (Contracted
    // into a fused operation one product would not be rounded, and each lane's share off by up to half a
    // unit of c: entropies of 2048 classes were off by 2.4e-5 at logits around 1000 and 3e-3 around
    // 100000; they are off by 9e-7 at any offset.)
    __device__ __forceinline__ void rise(float m)
    {
        if (!(m > top)) return;
        const float d = fmaxf(__fsub_rn(__fmul_rn(top, kLog2e), __fmul_rn(m, kLog2e)), -300.0f), e = exp2_fast(d);
        t = (t + d * s) * e;
        s *= e;
        top = m;
    }
};

// A thread's sums, two elements at a time: five instructions an element, so that memory and not
// their issue bounds the forward pass.
struct PairSums {
    float top;
    float2 s, t;

    __device__ __forceinline__ void clear()
    {
        top = kLpStart;
        s = t = make_float2(0.0f, 0.0f);
    }
    __device__ __forceinline__ void rise(float m)
    {
        if (!(m > top)) return;
        Sums a{top, s.x, t.x}, b{top, s.y, t.y};
        a.rise(m);
        b.rise(m);
        top = m;
        s = make_float2(a.s, b.s);
        t = make_float2(a.t, b.t);
    }
    __device__ __forceinline__ void add(float2 x)
    {
        const float c = -__fmul_rn(top, kLog2e);
        float2 y = __ffma2_rn(x, make_float2(kLog2e, kLog2e), make_float2(c, c));
        y = make_float2(max_nan(y.x, -200.0f), max_nan(y.y, -200.0f));      // (-inf times 0 would be a NaN)
        const float2 e = make_float2(exp2_fast(y.x), exp2_fast(y.y));
        s = __fadd2_rn(s, e);
        t = __ffma2_rn(y, e, t);
    }
    __device__ __forceinline__ Sums total() const { return Sums{top, s.x + s.y, t.x + t.y}; }
};

// the sums of 32 lanes, in every lane
__device__ __forceinline__ Sums warp_join(Sums a)
{
    float m = a.top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    a.rise(m);
    a.s = warp_sum(a.s);
    a.t = warp_sum(a.t);
    return a;
}

// The same sums for rows far from 0, in natural units: x - top is exact enough anywhere. All lanes of a warp, the whole row.
struct FarSums {
    float top, s, t;             // t: of (x - top) exp(x - top)
};

template <typename T>
__device__ __noinline__ FarSums far_sums(const T* row, int classes)
{
    const int lane = threadIdx.x & 31;
    FarSums f{-INFINITY, 0.0f, 0.0f};
    for (int c = lane; c < classes; c += 32) f.top = fmaxf(f.top, to_f32(row[c]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) f.top = fmaxf(f.top, __shfl_xor_sync(0xffffffffu, f.top, o));
    for (int c = lane; c < classes && f.top > -INFINITY; c += 32) {
        const float d = max_nan(to_f32(row[c]) - f.top, -1000.0f), e = expf(d);
        f.s += e;
        f.t += d * e;
    }
    f.s = warp_sum(f.s);
    f.t = warp_sum(f.t);
    return f;
}

// ------------------------------------------------------------- a warp's alternatives
//
// Lane i holds the i-th best of what the warp has taken in. Elements that come before `low` go
// to a buffer of 64 in shared memory; when 2 k + 2 of them (32 at most) are there, flush() brings
// them to the list, and its k-th best becomes `low`. (For 4 of 32768 in random order that is 3
// times a row, with 22 vectors looked at; waiting for 32 elements it was 32 vectors. 4096 x 32768
// bf16: 73 us with 4 alternatives, 75 us with sorts only.) The first `low` is the k-th largest of the
// lanes' largest elements of the first round, of all warps that share the row's part: at least k
// elements are no smaller, and in random order few more than k of that round and of each
// following one come before it. (With each warp's own, and the largest of them, 1200 x 32768 bf16
// with 8 and 32 alternatives took 34 and 83 us instead of 30 and 51.)
struct FirstLows {
    alignas(16) float v[kLpWarps * kLpMaxTop];
    float low;
};

struct Alternatives {
    Key best, low;
    float low_value;             // the smallest value that may still come before `low`
    int count;
    bool sorted;                 // the list holds elements
    Key* buf;

    __device__ __forceinline__ void clear(Key* b)
    {
        best = low = 0;
        low_value = -INFINITY;
        count = 0;
        sorted = false;
        buf = b;
    }
    // the first `low` of a warp that has a row for itself, from its lanes' largest elements in order
    __device__ __forceinline__ void first_low(float m, int k)
    {
        from_value(__shfl_sync(0xffffffffu, in_order(m), k - 1));
    }
    // of a block that shares a row: the k-th of its lanes'. All threads.
    __device__ __forceinline__ void first_low_of_block(float m, int k, int warp, FirstLows* f)
    {
        const int lane = threadIdx.x & 31;
        m = in_order(m);
        if (lane < k) f->v[warp * k + lane] = m;
        __syncthreads();
        if (lane < k) {
            const int me = warp * k + lane;
            int before = 0;
            for (int j = 0; j < kLpWarps * k; j += 4) {
                const float4 o = *reinterpret_cast<const float4*>(f->v + j);
                before += (o.x > m || (o.x == m && j < me)) + (o.y > m || (o.y == m && j + 1 < me)) +
                          (o.z > m || (o.z == m && j + 2 < me)) + (o.w > m || (o.w == m && j + 3 < me));
            }
            if (before == k - 1) f->low = m;
        }
        __syncthreads();
        from_value(f->low);
    }
    // the i-th largest of the lanes' m, in lane i (a NaN counts as lowest here)
    static __device__ __forceinline__ float in_order(float m)
    {
        const int lane = threadIdx.x & 31;
        if (m != m) m = -INFINITY;
#pragma unroll
        for (int size = 2; size <= 32; size *= 2)
#pragma unroll
            for (int j = size / 2; j > 0; j /= 2) {
                const float o = __shfl_xor_sync(0xffffffffu, m, j);
                m = ((lane & j) == 0) == ((lane & size) == 0) ? fmaxf(m, o) : fminf(m, o);
            }
        return m;
    }
    __device__ __forceinline__ void from_value(float v)
    {
        low_value = v;
        low = (Key)value_order(v) << 32;     // (every element of that value comes before it)
    }
    // the better of a lane's and its partner's (lane ^ j), or the worse
    static __device__ __forceinline__ Key exchange(Key a, int j, bool better)
    {
        const Key o = __shfl_xor_sync(0xffffffffu, a, j);
        return (a > o) == better ? a : o;
    }
    // 32 sorted elements, one to a lane
    __device__ __forceinline__ void merge(Key a, int k)
    {
        const int lane = threadIdx.x & 31;
        const Key r = __shfl_sync(0xffffffffu, a, 31 - lane);
        best = r > best ? r : best;
#pragma unroll
        for (int j = 16; j > 0; j /= 2) best = exchange(best, j, (lane & j) == 0);
        take_low(k);
    }
    __device__ __forceinline__ void take_low(int k)
    {
        low = __shfl_sync(0xffffffffu, best, k - 1);
        // Later elements of the same value have higher indexes: only larger ones come before it. (4096 x
        // 32768 bf16 with 4 alternatives, all elements equal: 60 us, 388 with equal ones looked at;
        // half of them masked 83, 243.)
        low_value = low ? key_value(((low >> 32) + 1) << 32) : -INFINITY;
        sorted = true;
    }
    __device__ __forceinline__ void merge_unsorted(Key a, int k)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int size = 2; size <= 32; size *= 2)
#pragma unroll
            for (int j = size / 2; j > 0; j /= 2) a = exchange(a, j, ((lane & j) == 0) == ((lane & size) == 0));
        merge(a, k);
    }
    // The k best of lists and buffer. Where they fit a warp each lane counts the elements before its
    // own: as many broadcast reads as elements, where a sort is 40 shuffles one after another.
    __device__ __forceinline__ void flush(int k)
    {
        const int lane = threadIdx.x & 31;
        if (count + k <= 32) {
            if (lane < k) buf[count + lane] = best;
            __syncwarp();
            const int n = count + k;
            const Key a = lane < n ? buf[lane] : 0;
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += buf[j] > a;
            if (a) buf[32 + rank] = a;
            const int there = __popc(__ballot_sync(0xffffffffu, a != 0));
            __syncwarp();
            best = lane < min(k, there) ? buf[32 + lane] : 0;
            __syncwarp();
            count = 0;
            take_low(k);
            return;
        }
        __syncwarp();
        const Key a = lane < count ? buf[lane] : 0, more = buf[32 + lane];
        __syncwarp();
        buf[lane] = more;
        count = max(count - 32, 0);
        merge_unsorted(a, k);
    }
    // all lanes, each with an element of its own (take false: none)
    __device__ __forceinline__ void offer(Key a, bool take, int k)
    {
        take = take && a > low;
        const unsigned m = __ballot_sync(0xffffffffu, take);
        if (!m) return;
        if (take) buf[count + __popc(m & ((1u << (threadIdx.x & 31)) - 1u))] = a;
        count += __popc(m);
        if (count >= min(32, 2 * k + 2)) flush(k);
    }
    // leaves everything in the buffer, -> how many (32 at most)
    __device__ __forceinline__ int gather(int k)
    {
        const int lane = threadIdx.x & 31;
        if (!sorted) return count;
        if (count + k > 32) flush(k);
        if (lane < k) buf[count + lane] = best;
        return count + k;
    }
};

// The k best of several buffers' elements, counts[i] (or each) of them in buffer i, into `out` (of
// 32 zeros): warp i takes buffer i, each thread counts the elements before its own.
__device__ __forceinline__ void rank_all(const Key (*buf)[64], int buffers, const int* counts, int each, int k, Key* out)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp >= buffers) return;
    const int n = counts ? counts[warp] : each;
    const Key mine = lane < n ? buf[warp][lane] : 0;
    if (!__any_sync(0xffffffffu, mine != 0)) return;
    int rank = 0;
    for (int w = 0; w < buffers; ++w) {
        const int m = counts ? counts[w] : each;
        for (int j = 0; j < m; ++j) rank += buf[w][j] > mine;
    }
    if (mine && rank < k) out[rank] = mine;
}

// The q-th lane of a set (-1: none), and in `from` its first four.
__device__ __forceinline__ int four_lanes(unsigned& from, int q)
{
    unsigned mine = from, rest = from;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (q > i) mine &= mine - 1;
        rest &= rest - 1;
    }
    from ^= rest;
    return __ffs(mine) - 1;
}

// Offers the elements of a warp's vectors that may be alternatives: v[u] of this lane starts at
// element first + u pitch, its elements are `skip` apart. ALL: every vector, not only those whose
// largest element is no smaller than `low` (a NaN is in no largest).
template <bool ALL, typename T, int UNROLL>
__device__ __forceinline__ void offer_vectors(const Vec<T> (&v)[UNROLL], int first, int pitch, int skip, int end, int k,
                                              Alternatives& alt)
{
    constexpr int PER = Vec<T>::kPer;
    const int lane = threadIdx.x & 31;
    unsigned pending = 0;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
        if (ALL || v[u].largest() >= alt.low_value) pending |= 1u << u;
    // four lanes' first such vectors at a time, their elements side by side; beyond the end are none
    for (unsigned from; (from = __ballot_sync(0xffffffffu, pending != 0)) != 0;) {
        const int src = four_lanes(from, lane / PER), u = __ffs(pending) - 1;
        Vec<T> w = v[0], b;
#pragma unroll
        for (int q = 1; q < UNROLL; ++q)
            if (u == q) w = v[q];
        const int at = src & 31;
        b.raw = make_uint4(__shfl_sync(0xffffffffu, w.raw.x, at), __shfl_sync(0xffffffffu, w.raw.y, at),
                           __shfl_sync(0xffffffffu, w.raw.z, at), __shfl_sync(0xffffffffu, w.raw.w, at));
        const int i = __shfl_sync(0xffffffffu, first + u * pitch, at) + (lane & (PER - 1)) * skip;
        if (from >> lane & 1u) pending &= pending - 1;
        alt.offer(make_key(b.element(lane & (PER - 1)), i), src >= 0 && lane < 4 * PER && i < end, k);
    }
}

constexpr int kLpUnroll = 4;         // vectors of a lane in a round

template <typename T>
__device__ __forceinline__ float largest_of(const Vec<T> (&v)[kLpUnroll])
{
    return fmaxf(fmaxf(v[0].largest(), v[1].largest()), fmaxf(v[2].largest(), v[3].largest()));
}

template <typename T>
__device__ __forceinline__ void add_vectors(PairSums& sums, const Vec<T> (&v)[kLpUnroll])
{
    constexpr int PER = Vec<T>::kPer;
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) {
        float f[PER];
        v[u].get(f);
#pragma unroll
        for (int j = 0; j < PER; j += 2) sums.add(make_float2(f[j], f[j + 1]));
    }
}

// A round of elements [base, end) of a row for thread `at` of `threads`. A vector's elements are
// neighbours (VEC; base on 16 bytes), or a warp's width apart where rows start anywhere: a warp's
// single loads are still consecutive.
template <bool VEC, typename T>
__device__ __forceinline__ int load_round(Vec<T> (&v)[kLpUnroll], const T* __restrict__ row, int base, int end, int at,
                                          int threads)
{
    constexpr int PER = Vec<T>::kPer, skip = VEC ? 1 : 32;
    const int lane = threadIdx.x & 31, first = base + (at - lane) * PER + (VEC ? lane * PER : lane);
#pragma unroll
    for (int u = 0; u < kLpUnroll; ++u) {
        const int c = first + u * threads * PER;
        if (VEC && c + PER <= end) {
            v[u].raw = __ldcs(reinterpret_cast<const uint4*>(row + c));
        } else {
            float f[PER];
#pragma unroll
            for (int j = 0; j < PER; ++j) f[j] = c + j * skip < end ? to_f32(row[c + j * skip]) : -INFINITY;
            v[u].set(f);                 // exact: the values came from T
        }
    }
    return first;
}

// The alternatives of a warp's part of a row that holds a NaN (or an infinity that made one).
template <typename T, bool VEC>
__device__ __noinline__ void scan_every(const T* row, int begin, int end, int at, int threads, int k, Alternatives* alt)
{
    constexpr int PER = Vec<T>::kPer;
    Alternatives a;
    a.clear(alt->buf);
    __syncwarp();
    for (int base = begin; base < end; base += threads * PER * kLpUnroll) {
        Vec<T> v[kLpUnroll];
        const int first = load_round<VEC>(v, row, base, end, at, threads);
        offer_vectors<true>(v, first, threads * PER, VEC ? 1 : 32, end, k, a);
    }
    *alt = a;
}
template <typename T, bool VEC>
__device__ __forceinline__ void scan_again(const T* row, int begin, int end, int at, int threads, int k, Alternatives& alt)
{
    Alternatives a;
    a.buf = alt.buf;
    scan_every<T, VEC>(row, begin, end, at, threads, k, &a);
    alt = a;
}

// Elements [begin, end) of a row for thread `at` of `threads`. lows: the block's first
// thresholds, where its warps share the row (then every warp passes here).
template <typename T, bool TOP, bool VEC>
__device__ __forceinline__ Sums scan(const T* __restrict__ row, int begin, int end, int at, int threads, int k,
                                     Alternatives& alt, FirstLows* lows)
{
    constexpr int PER = Vec<T>::kPer;
    PairSums sums;
    sums.clear();
    // (classes are at most 2^30: no index overflows)
    for (int base = begin; base < end; base += threads * PER * kLpUnroll) {
        Vec<T> v[kLpUnroll];
        const int first = load_round<VEC>(v, row, base, end, at, threads);
        const float m = largest_of(v);
        sums.rise(m);
        if (TOP && base == begin) {
            if (lows) alt.first_low_of_block(m, k, at >> 5, lows);
            else alt.first_low(m, k);
        }
        add_vectors(sums, v);
        if (TOP && __any_sync(0xffffffffu, m >= alt.low_value))
            offer_vectors<false>(v, first, threads * PER, VEC ? 1 : 32, end, k, alt);
    }
    const Sums s = sums.total();
    if (TOP && __any_sync(0xffffffffu, s.s != s.s)) scan_again<T, VEC>(row, begin, end, at, threads, k, alt);
    return s;
}

struct LpOut {
    float *logp, *entropy, *lse;
    int32_t* top_ids;
    float* top_logp;
};

// the row's results from its sums and (lane i: the i-th) alternatives; one warp
template <typename T, bool TOP>
__device__ __forceinline__ void write_row(const T* row, const int32_t* targets, int64_t r, int classes, int k,
                                          const Sums& a, const Alternatives& alt, const LpOut& o, int* err)
{
    const int lane = threadIdx.x & 31;
    float lse, entropy, top, ls;
    bool none = false, far = false;
    if (!(a.s < 0.5f) && (a.top <= kLpReach || a.s != a.s)) {
        const float l2 = log2f(a.s);
        top = a.top;
        ls = l2 * kLn2;
        lse = a.top + ls;
        entropy = (l2 - a.t / a.s) * kLn2;
    } else {
        const FarSums f = far_sums(row, classes);
        none = f.top == -INFINITY;
        far = true;
        top = f.top;
        ls = logf(f.s);
        lse = none ? -INFINITY : f.top + ls;
        entropy = none ? 0.0f : ls - f.t / f.s;
    }
    // counted from top as the sums were, whose c is rounded; far below it that does not matter
    auto log_p = [&](float x) {
        const float d = x - top;
        if (none) return -INFINITY;
        return (far || d < -kLpReach ? d : fmaf(x, kLog2e, -__fmul_rn(top, kLog2e)) * kLn2) - ls;
    };
    if (lane == 0) {
        if (o.lse) o.lse[r] = lse;
        if (o.entropy) o.entropy[r] = entropy;
        if (o.logp) {
            const int t = targets[r];
            if (t < -1 || t >= classes) raise_device_error(err, ITO_ERR_ARG);
            o.logp[r] = t < 0 || t >= classes ? 0.0f : log_p(to_f32(row[t]));
        }
    }
    if (TOP && lane < k) {
        o.top_ids[r * k + lane] = key_index(alt.best);
        o.top_logp[r * k + lane] = log_p(key_value(alt.best));
    }
}

// Short rows and rows enough: a warp to a row, the warps of all blocks with nearly as many rows.
// The loads are ahead of the work: each warp keeps a ring of kLpSlots rounds in shared memory,
// filled by bulk copies, and the vectors that may hold alternatives are read again there, four at
// a time. A row is taken from the 16-byte boundary before it, `lead` elements early; its first and
// last elements that fill no vector are loaded singly. 4096 x 32768 bf16 with 4
// alternatives: 60 us (without any 45, the rows' bytes at the device's copy rate 40), 80 with loads
// to registers and shuffles; rows of 32001 63 us, 104 with single loads. What bounds it: 11500
// instructions a warp and row, 8500 of them for the sums.
// A block is of few warps with alternatives, so that an SM holds 28 at 72 registers (32 at 64
// spill: 73 us), else of 8 with 32 to an SM. Either way shared memory or registers let no SM take
// more blocks than its share of the grid, while the previous launch's end: 75 us where they did.
// After a wait that runs out (mbar_wait, ITO_ERR_TIMEOUT) a warp writes no more rows and leaves when its
// copies under way have landed.
constexpr int ring_warps(bool top) { return top ? 4 : 8; }         // of a block
constexpr int ring_blocks(bool top) { return top ? 7 : 4; }        // of an SM
constexpr int kLpSlots = 3, kLpRound = 32 * kLpUnroll * 16;      // bytes of a round

template <typename T>
__device__ __forceinline__ int elements_before(const T* p)
{
    return (int)(reinterpret_cast<uintptr_t>(p) & 15u) / (int)sizeof(T);
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(ring_warps(TOP) * 32, ring_blocks(TOP))
    k_logprobs_ring(const T* __restrict__ x, int64_t ld, const int32_t* __restrict__ targets, int64_t rows,
                    int classes, int k, const LpOut o, int* __restrict__ err)
{
    constexpr int WARPS = ring_warps(TOP), PER = Vec<T>::kPer, EACH = kLpRound / (int)sizeof(T);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Key buf[WARPS][TOP ? 64 : 1];
    __shared__ uint64_t full[WARPS][kLpSlots];
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* const ring = smem + warp * (kLpSlots * kLpRound);
    if (threadIdx.x == 0) abort_flag = 0;
    if (lane == 0) {
        for (int s = 0; s < kLpSlots; ++s) mbar_init(&full[warp][s], 1);
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const int64_t step = (int64_t)gridDim.x * WARPS;
    int64_t r = (int64_t)warp * gridDim.x + blockIdx.x, ahead = r;
    int ahead_base = 0;
    auto fetch = [&](int s) {            // the next round of this warp's rows
        if (ahead >= rows) return;
        const T* const row = x + ahead * ld;
        const int lead = elements_before<T>(row), end = min(ahead_base + EACH, classes + lead) / PER * PER;
        const int from = ahead_base || !lead ? ahead_base : PER;
        const uint32_t bytes = (uint32_t)(max(end - from, 0) * (int)sizeof(T));
        if (lane == 0) {
            mbar_arrive_expect_tx(&full[warp][s], bytes);
            if (bytes) bulk_load(ring + s * kLpRound + (from - ahead_base) * (int)sizeof(T), row - lead + from, bytes, &full[warp][s]);
        }
        ahead_base += EACH;
        if (ahead_base >= classes + lead) ahead_base = 0, ahead += step;
    };
    for (int s = 0; s < kLpSlots; ++s) fetch(s);
    int slot = 0;
    uint32_t phase = 0;
    for (; r < rows; r += step) {
        const T* const row = x + r * ld;
        Alternatives alt;
        alt.clear(buf[warp]);
        PairSums sums;
        sums.clear();
        const int lead = elements_before<T>(row), end = classes + lead;
        for (int base = 0; base < end; base += EACH) {
            if (!__all_sync(0xffffffffu, mbar_wait(&full[warp][slot], phase, &abort_flag, err))) {
                if (lane == 0) ring_landed(full[warp], kLpSlots, RingPlace{slot, phase}, kLpSlots);
                return;
            }
            uint8_t* const at = ring + slot * kLpRound;
            Vec<T> v[kLpUnroll];
            float m[kLpUnroll];
#pragma unroll
            for (int u = 0; u < kLpUnroll; ++u) v[u].raw = *reinterpret_cast<const uint4*>(at + (u * 32 + lane) * 16);
            if (base + EACH > end || (base == 0 && lead)) {
                // what is no whole vector, and nothing before the row or beyond it
#pragma unroll
                for (int u = 0; u < kLpUnroll; ++u) {
                    const int c = base + (u * 32 + lane) * PER;
                    float f[PER];
                    if (c >= lead && c + PER <= end) continue;
#pragma unroll
                    for (int j = 0; j < PER; ++j) f[j] = c + j >= lead && c + j < end ? to_f32(row[c + j - lead]) : -INFINITY;
                    v[u].set(f);
                    if (TOP) *reinterpret_cast<uint4*>(at + (u * 32 + lane) * 16) = v[u].raw;
                }
                if (TOP) fence_proxy_async_smem();
            }
#pragma unroll
            for (int u = 0; u < kLpUnroll; ++u) m[u] = v[u].largest();
            const float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
            sums.rise(most);
            if (TOP && base == 0) alt.first_low(most, k);
            add_vectors(sums, v);
            __syncwarp();
            if (TOP && __any_sync(0xffffffffu, most >= alt.low_value)) {
                unsigned pending = 0;    // this lane's vectors to look at closer
#pragma unroll
                for (int u = 0; u < kLpUnroll; ++u) pending |= m[u] >= alt.low_value ? 1u << u : 0u;
                // four lanes' vectors at a time, their elements from shared memory
                for (unsigned from; (from = __ballot_sync(0xffffffffu, pending != 0)) != 0;) {
                    const int src = four_lanes(from, lane / PER), at_src = src & 31;
                    const int u = __shfl_sync(0xffffffffu, __ffs(pending) - 1, at_src);
                    if (from >> lane & 1u) pending &= pending - 1;
                    const bool there = src >= 0 && lane < 4 * PER;
                    const int e = (u * 32 + at_src) * PER + (lane & (PER - 1));
                    float f = 0.0f;
                    if (there) f = to_f32(reinterpret_cast<const T*>(at)[e]);
                    const int i = base + e - lead;
                    alt.offer(make_key(f, i), there && i >= 0 && i < classes, k);
                }
                __syncwarp();
            }
            fetch(slot);
            if (++slot == kLpSlots) slot = 0, phase ^= 1;
        }
        const Sums a = sums.total();
        if (TOP && __any_sync(0xffffffffu, a.s != a.s)) scan_again<T, false>(row, 0, classes, lane, 32, k, alt);
        if (TOP && alt.count) alt.flush(k);
        write_row<T, TOP>(row, targets, r, classes, k, warp_join(a), alt, o, err);
    }
}

// Longer rows: a cluster of blocks to a row (of one block, where there are rows enough), each
// with a stretch of it. The warps' sums and alternatives meet in their block's shared memory, the
// blocks' in the first one's, read across the cluster.
template <typename T, bool TOP, bool VEC>
__global__ void __launch_bounds__(kLpWarps * 32, 4)
    k_logprobs_long(const T* __restrict__ x, int64_t ld, const int32_t* __restrict__ targets, int64_t rows,
                    int classes, int k, int parts, int stretch, const LpOut o, int* __restrict__ err)
{
    static_assert(kLpCluster <= kLpWarps, "a warp to each block of the cluster");
    __shared__ Sums sums[kLpWarps];
    __shared__ FirstLows lows;
    __shared__ int counts[kLpWarps];
    __shared__ Key buf[TOP ? kLpWarps : 1][64], list[2][32];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = parts > 1 ? (int)cluster_ctarank() : 0;
    const int begin = min(classes, part * stretch), end = min(classes, begin + stretch);
    for (int64_t r = blockIdx.x / parts; r < rows; r += gridDim.x / parts) {
        Alternatives alt;
        alt.clear(buf[TOP ? warp : 0]);
        if (TOP && warp < 2) list[warp][lane] = 0;
        Sums a = warp_join(scan<T, TOP, VEC>(x + r * ld, begin, end, threadIdx.x, kLpWarps * 32, k, alt, &lows));
        if (TOP) {
            const int n = alt.gather(k);
            if (lane == 0) counts[warp] = n;
        }
        if (lane == 0) sums[warp] = a;
        __syncthreads();
        if (warp == 0) a = warp_join(lane < kLpWarps ? sums[lane] : Sums{kLpStart, 0.0f, 0.0f});
        if (TOP) {
            rank_all(buf, kLpWarps, counts, 0, k, list[0]);
            __syncthreads();
        }
        if (parts > 1) {
            if (threadIdx.x == 0) sums[0] = a;
            cluster_sync();
            if (part == 0) {
                if (TOP && warp < parts) {
                    Key v = 0;
                    if (lane < k)
                        asm volatile("ld.shared::cluster.u64 %0, [%1];"
                                     : "=l"(v) : "r"(mapa_shared(smem_u32(&list[0][lane]), warp)) : "memory");
                    buf[warp][lane] = v;
                }
                if (warp == 0) {
                    const uint32_t sa = mapa_shared(smem_u32(&sums[0]), lane < parts ? lane : 0);
                    Sums q;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(q.top) : "r"(sa) : "memory");
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(q.s) : "r"(sa + 4) : "memory");
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(q.t) : "r"(sa + 8) : "memory");
                    if (lane >= parts) q.clear();
                    a = warp_join(q);
                }
                if (TOP) {
                    __syncthreads();
                    rank_all(buf, parts, nullptr, k, k, list[1]);
                    __syncthreads();
                }
            }
            cluster_sync();              // the first block has read the others' shared memory
        }
        if (part == 0 && warp == 0) {
            alt.best = list[parts > 1][lane];
            write_row<T, TOP>(x + r * ld, targets, r, classes, k, a, alt, o, err);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------- the gradient
//
// A block takes a stretch of a row (or its warps a row each, where rows are short). Where the
// row and its gradient start equally far from a 16-byte boundary, the elements up to the first
// boundary and after the last go alone and the rest in 16-byte vectors.

//
// log p = x - lse is as good as lse, whose own rounding grows with it: from 2^16 on (rows of
// masks of the type's lowest value) the row's sums are taken again, and log p is
// (x - top) - log s. (Not where the gradient replaces the logits of a row that several blocks
// share: there the row is being overwritten.)
struct LpRow {
    float top, ls, g, gh, h;
    int t;
};
constexpr float kLpFar = 65536.0f;

// dx_j: the factor of p is one sum, so p (which may lie below the normal range) is rounded once.
// A p of 0 takes no part: the log p of a class masked with the type's lowest value, times a
// g_H above 1, would be infinite.
__device__ __forceinline__ float lp_slope(const LpRow& w, float x, int c)
{
    float d = c == w.t ? w.g : 0.0f;
    const float lp = (x - w.top) - w.ls, p = __expf(lp);
    if (x != -INFINITY && p != 0.0f) d -= p * (w.g + w.gh * (lp + w.h));
    return d;
}

constexpr int kLpStretch = 8192;     // elements of a row that a block takes, at most

template <typename T>
__global__ void __launch_bounds__(256, 4)
    k_logprobs_bwd(const T* __restrict__ x, int64_t ld, const int32_t* __restrict__ targets,
                   const float* __restrict__ lse, const float* __restrict__ entropy, int64_t rows, int classes,
                   const float* __restrict__ g_logp, const float* __restrict__ g_entropy, T* __restrict__ dx,
                   int64_t ldd, int per_warp, int stretches, int* __restrict__ err)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int PER = Vec<T>::kPer, UNROLL = 4;
    const int at = per_warp ? threadIdx.x & 31 : threadIdx.x, threads = per_warp ? 32 : 256;
    const int64_t work = per_warp ? rows : rows * stretches;
    const int64_t first = per_warp ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = per_warp ? (int64_t)gridDim.x * 8 : gridDim.x;
    for (int64_t i = first; i < work; i += step) {
        const int64_t r = per_warp ? i : i / stretches;
        const float z = lse[r];
        LpRow w;
        w.top = z;
        w.ls = 0.0f;
        w.t = targets ? targets[r] : -1;
        if (w.t < -1 || w.t >= classes) {
            if (at == 0) raise_device_error(err, ITO_ERR_ARG);
            w.t = -1;
        }
        w.g = w.t >= 0 && g_logp ? g_logp[r] : 0.0f;
        w.gh = g_entropy ? g_entropy[r] : 0.0f;
        w.h = g_entropy ? entropy[r] : 0.0f;
        const T* xr = x + r * ld;
        T* dr = dx + r * ldd;
        if (fabsf(z) >= kLpFar && fabsf(z) < INFINITY && (stretches == 1 || dx != x)) {
            const FarSums f = far_sums(xr, classes);    // each warp for itself
            w.top = f.top;
            w.ls = logf(f.s);
            if (!per_warp) __syncthreads();             // (the row is the block's; dx may be x)
        }
        const int lead_x = (int)((16 - (reinterpret_cast<uintptr_t>(xr) & 15)) & 15) / (int)sizeof(T);
        const int lead_d = (int)((16 - (reinterpret_cast<uintptr_t>(dr) & 15)) & 15) / (int)sizeof(T);
        const int lead = min(lead_x, classes);
        const bool vec = lead_x == lead_d;
        const int64_t s = per_warp ? 0 : i - r * stretches;
        // stretch s of the row counts from the first boundary; the first one takes the lead too
        const int64_t b0 = lead + s * kLpStretch;
        const int begin = (int)min((int64_t)classes, b0);
        const int end = per_warp || s == stretches - 1 ? classes : (int)min((int64_t)classes, b0 + kLpStretch);
        if (z == -INFINITY) {
            for (int c = (s == 0 ? 0 : begin) + at; c < end; c += threads) dr[c] = from_f32<T>(0.0f);
            continue;
        }
        if (s == 0 && at < lead) dr[at] = from_f32<T>(lp_slope(w, to_f32(xr[at]), at));
        int c = begin;
        if (vec) {
            const int whole = begin + (end - begin) / PER * PER;
            for (; c < whole; c += threads * PER * UNROLL) {
                Vec<T> v[UNROLL];
#pragma unroll
                for (int u = 0; u < UNROLL; ++u) {
                    const int k = c + (u * threads + at) * PER;
                    if (k < whole) v[u].raw = __ldcs(reinterpret_cast<const uint4*>(xr + k));
                }
#pragma unroll
                for (int u = 0; u < UNROLL; ++u) {
                    const int k = c + (u * threads + at) * PER;
                    if (k >= whole) continue;
                    float f[PER];
                    v[u].get(f);
#pragma unroll
                    for (int j = 0; j < PER; ++j) f[j] = lp_slope(w, f[j], k + j);
                    v[u].set(f);
                    __stcs(reinterpret_cast<uint4*>(dr + k), v[u].raw);
                }
            }
            c = whole;
        }
#pragma unroll 4
        for (int k = c + at; k < end; k += threads) dr[k] = from_f32<T>(lp_slope(w, to_f32(xr[k]), k));
    }
}

static int check_lp(const void* x, int64_t ld, int type, int64_t rows, int classes)
{
    if (!x) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    if (!type_known(type)) return set_error(ITO_ERR_ARG, "unknown type");
    if (rows < 1 || classes < 1) return set_error(ITO_ERR_SHAPE, "sizes must be >= 1");
    if (rows > (int64_t(1) << 40) || classes > (1 << 30)) return set_error(ITO_ERR_SHAPE, "rows above 2^40 or classes above 2^30");
    if (rows > 1 && ld < classes) return set_error(ITO_ERR_SHAPE, "row stride below classes");
    if (!aligned_to(x, type_bytes(type))) return set_error(ITO_ERR_ARG, "misaligned pointer");
    return ITO_OK;
}

template <typename T, bool TOP>
static int run_fwd(const void* xp, int64_t ld, const int32_t* targets, int64_t rows, int classes, int k,
                   const LpOut& o, int* err, cudaStream_t s)
{
    const T* x = static_cast<const T*>(xp);
    const int sms = num_sms();
    // A warp to a row up to four vectors a lane, or with eight rows to an SM: no warp waits for
    // another then. bf16 with 0, 1, 4, 8 alternatives, against a block to a row:
    // 2500 x 32768 31, 44, 49, 53 us, 36, 46, 53, 61; 1500 x 5000 5, 9, 10, 12 us, 9, 14, 17, 21.
    // Fewer rows leave too few loads in flight (1200 x 32768 18, 29, 32, 35 us, 17, 22, 26, 30).
    const int round = 32 * Vec<T>::kPer * kLpUnroll;
    if (classes <= round || rows >= 8 * sms) {
        // (a block's warps take rows a grid apart, so SMs differ by a row at most)
        const unsigned grid = (unsigned)std::min(rows, (int64_t)ring_blocks(TOP) * sms);
        const auto kernel = k_logprobs_ring<T, TOP>;
        constexpr int smem = ring_warps(TOP) * kLpSlots * kLpRound;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return set_error(ITO_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(cudaGetLastError()));
        launch_pdl(kernel, grid, ring_warps(TOP) * 32, smem, s, x, ld, targets, rows, classes, k, o, err);
        return launch_status("log probabilities");
    }
    // blocks of a row: enough that all rows' blocks occupy the SMs, each with a round of loads at least
    int parts = 1;
    while (parts < kLpCluster && rows * parts * 2 <= 2 * sms && classes / (2 * parts) >= kLpWarps * round / 4) parts *= 2;
    const int stretch = ((classes + parts - 1) / parts + 15) / 16 * 16;
    const int64_t most = (int64_t)sms * 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(std::min(rows * parts, most) / parts * parts));
    cfg.blockDim = dim3(kLpWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = parts;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = parts > 1 ? 2 : 1;
    const cudaError_t e =
        rows_vec(x, ld, sizeof(T), rows)
            ? cudaLaunchKernelEx(&cfg, k_logprobs_long<T, TOP, true>, x, ld, targets, rows, classes, k, parts, stretch, o, err)
            : cudaLaunchKernelEx(&cfg, k_logprobs_long<T, TOP, false>, x, ld, targets, rows, classes, k, parts, stretch, o, err);
    return e == cudaSuccess ? ITO_OK : set_error(ITO_ERR_CUDA, "log probabilities launch: %s", cudaGetErrorString(e));
}

template <typename T>
static int run_fwd_any(const void* x, int64_t ld, const int32_t* targets, int64_t rows, int classes, int k,
                       const LpOut& o, int* err, cudaStream_t s)
{
    if (k) return run_fwd<T, true>(x, ld, targets, rows, classes, k, o, err, s);
    return run_fwd<T, false>(x, ld, targets, rows, classes, k, o, err, s);
}

template <typename T>
static int run_bwd(const void* x, int64_t ld, const int32_t* targets, const float* lse, const float* entropy,
                   int64_t rows, int classes, const float* g_logp, const float* g_entropy, void* dx, int64_t ldd,
                   int* err, cudaStream_t s)
{
    const int per_warp = classes <= 32 * Vec<T>::kPer * 4;
    const int stretches = (classes + kLpStretch - 1) / kLpStretch;
    const int64_t blocks = per_warp ? (rows + 7) / 8 : rows * stretches;
    launch_pdl(k_logprobs_bwd<T>, (unsigned)std::min<int64_t>(blocks, 1 << 30), 256, 0, s, static_cast<const T*>(x),
               ld, targets, lse, entropy, rows, classes, g_logp, g_entropy, static_cast<T*>(dx), ldd, per_warp,
               stretches, err);
    return launch_status("log probabilities");
}

}  // namespace ito

using namespace ito;

extern "C" {

int ito_token_logprobs_fwd(const void* logits, int64_t ld, int type, const int32_t* targets, int64_t rows, int classes,
                           int k, float* logp, float* entropy, float* lse, int32_t* top_ids, float* top_logp,
                           void* stream)
{
    const int r = check_lp(logits, ld, type, rows, classes);
    if (r) return r;
    if (k < 0 || k > kLpMaxTop) return set_error(ITO_ERR_ARG, "k must be in 0 .. %d", kLpMaxTop);
    if (k > classes) return set_error(ITO_ERR_SHAPE, "k above classes");
    if (k && (!top_ids || !top_logp)) return set_error(ITO_ERR_ARG, "NULL top_ids or top_logp");
    if (logp && !targets) return set_error(ITO_ERR_ARG, "logp needs targets");
    if (!k && !logp && !entropy && !lse) return set_error(ITO_ERR_ARG, "no output");
    if (!aligned_to(targets, 4) || !aligned_to(logp, 4) || !aligned_to(entropy, 4) || !aligned_to(lse, 4) ||
        !aligned_to(top_ids, 4) || !aligned_to(top_logp, 4))
        return set_error(ITO_ERR_ARG, "misaligned pointer");
    int* err = device_error_word();
    if (!err) return set_error(ITO_ERR_CUDA, "device error word unavailable");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const LpOut o{logp, entropy, lse, top_ids, top_logp};
    if (type == ITO_F32) return run_fwd_any<float>(logits, ld, targets, rows, classes, k, o, err, s);
    if (type == ITO_BF16) return run_fwd_any<__nv_bfloat16>(logits, ld, targets, rows, classes, k, o, err, s);
    return run_fwd_any<__half>(logits, ld, targets, rows, classes, k, o, err, s);
}

int ito_token_logprobs_bwd(const void* logits, int64_t ld, int type, const int32_t* targets, const float* lse,
                           const float* entropy, int64_t rows, int classes, const float* g_logp,
                           const float* g_entropy, void* dlogits, int64_t ldd, void* stream)
{
    const int r = check_lp(logits, ld, type, rows, classes);
    if (r) return r;
    if (!lse || !dlogits || (!g_logp && !g_entropy)) return set_error(ITO_ERR_ARG, "NULL tensor pointer");
    if (g_logp && !targets) return set_error(ITO_ERR_ARG, "g_logp needs targets");
    if (g_entropy && !entropy) return set_error(ITO_ERR_ARG, "g_entropy needs entropy");
    if (rows > 1 && ldd < classes) return set_error(ITO_ERR_SHAPE, "row stride below classes");
    if (!aligned_to(dlogits, type_bytes(type)) || !aligned_to(targets, 4) || !aligned_to(lse, 4) ||
        !aligned_to(entropy, 4) || !aligned_to(g_logp, 4) || !aligned_to(g_entropy, 4))
        return set_error(ITO_ERR_ARG, "misaligned pointer");
    int* err = device_error_word();
    if (!err) return set_error(ITO_ERR_CUDA, "device error word unavailable");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (type == ITO_F32)
        return run_bwd<float>(logits, ld, targets, lse, entropy, rows, classes, g_logp, g_entropy, dlogits, ldd, err, s);
    if (type == ITO_BF16)
        return run_bwd<__nv_bfloat16>(logits, ld, targets, lse, entropy, rows, classes, g_logp, g_entropy, dlogits,
                                      ldd, err, s);
    return run_bwd<__half>(logits, ld, targets, lse, entropy, rows, classes, g_logp, g_entropy, dlogits, ldd, err, s);
}

}  // extern "C"
