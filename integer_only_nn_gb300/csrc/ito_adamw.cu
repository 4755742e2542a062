// The AdamW step over many tensors, its moments held in 32 bits or in 8, in one launch for up to
// kAdamEntries tensors; with 8-bit moments and tensors of many chunks in two, their whole chunks and the rest.
//
//   m = b1 m + (1 - b1) g           v = b2 v + (1 - b2) g^2
//   w = w (1 - lr wd) - (m lr / (1 - b1^t)) / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Every operation is one IEEE operation in 32 bits, in this order (no contraction into fused
// multiply-adds), so a plain program that rounds after each operation gets the same bits.
//
// Moments in 8 bits: blocks of 128 consecutive elements of a tensor share a signed 8-bit
// exponent E, as the Blocked-DFP tensors do, and an element is a byte under it:
//   m: sign, 4 exponent bits, 3 mantissa bits:  +-2^(E - 15 + (c >> 3)) (1 + (c & 7) / 8)
//   v: 5 exponent bits, 3 mantissa bits:           2^(E - 31 + (c >> 3)) (1 + (c & 7) / 8)
// with c = 0 standing for zero, and E = -128 for a block that held an infinity or a NaN (all
// its elements read NaN). E is the exponent of the block's largest magnitude, rounded up to
// four significant bits, so that no element rounds past the largest code. The exponent field
// gives v 31 binades below the block's largest value, m 15: an element whose m survives has
// a v that survives, and a v above zero never becomes zero (its code is at least 1), so a
// small denominator cannot appear by rounding.
// A code's step is 1/8 to 1/16 of its value; nearest rounding would leave v where it stands,
// because (1 - b2) g^2 moves it by about 1/1000 a step. So both moments round
// stochastically: up with the probability of the part cut off, from a 32-bit mix of seed,
// step, tensor and element. The weight's own step uses the moments before they are rounded.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "ito_float.cuh"

namespace ito {

constexpr int kAdamBlock = 128;      // elements that share an exponent
constexpr int kAdamThreads = 256;
constexpr int kAdamChunk = 8192;     // elements a CTA takes

struct AdamEntry {
    float* w;
    const void* g;
    void* copy;
    void* m;
    void* v;
    int8_t* m_exp;
    int8_t* v_exp;
    int64_t n, from;        // elements; the first that this launch takes (a multiple of 128)
    uint32_t first_chunk;   // of this launch's chunks
    float decay;            // 1 - lr wd
    int32_t vec;            // the pointers allow four elements at a time
    uint32_t salt;          // the tensor's share of the rounding's key
};

constexpr int kAdamEntries = 44;     // of 88 bytes: the table is a kernel argument (4 KB at most)

struct AdamTable {
    int32_t n;
    AdamEntry e[kAdamEntries];
};

__device__ __forceinline__ int find_entry(const AdamTable& tab, uint32_t chunk)
{
    int lo = 0, hi = tab.n - 1;          // the tensor that holds the chunk
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.e[mid].first_chunk <= chunk) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// the tensor of a later chunk, from an earlier one's
__device__ __forceinline__ int next_entry(const AdamTable& tab, int i, uint32_t chunk)
{
    while (i + 1 < tab.n && tab.e[i + 1].first_chunk <= chunk) ++i;
    return i;
}

struct AdamConst {
    float b1, c1, b2, c2, eps, inv_sqrt_bc2, alpha, grad_scale;
    uint32_t key;
};

// ------------------------------------------------------------- 8-bit moments

// A 32-bit mix (multiply, fold the high half down; the multipliers are the fractional parts
// of the square roots of 2, 3 and 11): the low 20 bits round m, another 20 round v.
constexpr uint32_t kMixIndex = 0x6A09E667u;

// the element's index and the key, mixed: linear in the index's low half
__device__ __forceinline__ uint32_t round_key(uint32_t key, int64_t i)
{
    return (uint32_t)i * kMixIndex + (uint32_t)((uint64_t)i >> 32) * 0xBB67AE85u + key;
}

__device__ __forceinline__ void round_bits(uint32_t h, uint32_t& um, uint32_t& uv)
{
    h ^= h >> 16;
    h *= 0xBB67AE85u;
    h ^= h >> 15;
    h *= 0x6A09E667u;
    h ^= h >> 16;
    um = h & 0xFFFFFu;
    uv = (h * 0x510E527Fu) >> 12;
}

// What a byte's exponent and mantissa are added to under the exponent e (not -128).
template <bool SECOND>
__device__ __forceinline__ uint32_t moment_base(int e)
{
    return (uint32_t)(e + (SECOND ? 96 : 112)) << 23;
}

// the value of byte j of four codes
template <bool SECOND>
__device__ __forceinline__ float moment_value(uint32_t codes, int j, uint32_t base)
{
    // the byte at the top of a word; its exponent and mantissa belong four bits lower
    const uint32_t c = __byte_perm(codes, 0u, (uint32_t)j << 12 | 0x0444u);
    const uint32_t mag = SECOND ? c : c & 0x7F000000u;
    const uint32_t r = mag ? (mag >> 4) + base : 0u;
    return __uint_as_float(SECOND ? r : r | (c & 0x80000000u));
}

// the largest finite value that a code under the largest exponent stands for, 1.875 * 2^127
constexpr uint32_t kMomentTop = 0x7F700000u;

// the shared exponent of a block whose largest magnitude has these bits
template <bool SECOND>
__device__ __forceinline__ int moment_exponent(uint32_t top)
{
    if (top >= 0x7F800000u) return -128;
    const int e = (int)((min(top, kMomentTop) + 0xFFFFFu) >> 23) - 127;
    return max(e, SECOND ? -95 : -111);
}

// The code of x: its bits, counted from the lowest binade (base: moment_base), plus a random
// part of the step that is cut off. Below the lowest binade the count is negative and the code
// 0, or 1 for a v above zero. |x| is at most moment_top.
template <bool SECOND>
__device__ __forceinline__ uint32_t moment_code(float x, uint32_t base, uint32_t u)
{
    const uint32_t bits = __float_as_uint(x), mag = SECOND ? bits : bits & 0x7FFFFFFFu;
    const int c = (int)(mag - base + u) >> 20;
    if (SECOND) return (uint32_t)max(c, (int)min(mag, 1u));
    return c > 0 ? (uint32_t)c | (bits >> 24 & 128u) : 0u;
}

template <int N>
__device__ __forceinline__ void clamp_moments(float (&x)[N])
{
    const float top = __uint_as_float(kMomentTop);
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = fminf(fmaxf(x[j], -top), top);
}

// the larger magnitude; a NaN wins
__device__ __forceinline__ float larger(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

// ------------------------------------------------------------------- the step

__device__ __forceinline__ void adam_element(const AdamConst& k, float decay, float g, float& w, float& m, float& v)
{
    g = __fmul_rn(g, k.grad_scale);
    m = __fadd_rn(__fmul_rn(m, k.b1), __fmul_rn(g, k.c1));
    v = __fadd_rn(__fmul_rn(v, k.b2), __fmul_rn(__fmul_rn(g, g), k.c2));
    const float den = __fadd_rn(__fmul_rn(__fsqrt_rn(v), k.inv_sqrt_bc2), k.eps);
    w = __fsub_rn(__fmul_rn(w, decay), __fdiv_rn(__fmul_rn(m, k.alpha), den));
}

// Four consecutive elements (VEC: the pointers allow wide accesses) or four a warp apart of one
// block of 128 elements for each lane of a warp.
template <typename G, typename C, int BITS, bool VEC>
struct AdamPiece {
    float4 w, m32, v32;
    float g[4];
    uint32_t m8, v8;
    int em, ev;

    static __device__ __forceinline__ int64_t at(int64_t b, int lane, int j)
    {
        return VEC ? b + lane * 4 + j : b + j * 32 + lane;
    }
    __device__ __forceinline__ void load(const AdamEntry& e, int64_t b, int64_t end, int lane)
    {
        const G* gp = static_cast<const G*>(e.g);
        if (BITS == 8) {
            em = e.m_exp[b / kAdamBlock];
            ev = e.v_exp[b / kAdamBlock];
        }
        if (VEC && b + kAdamBlock <= end) {
            const int64_t i = b + lane * 4;
            w = *reinterpret_cast<const float4*>(e.w + i);
            if constexpr (sizeof(G) == 4) {
                const float4 q = __ldcs(reinterpret_cast<const float4*>(gp + i));
                g[0] = q.x; g[1] = q.y; g[2] = q.z; g[3] = q.w;
            } else {
                const uint2 q = __ldcs(reinterpret_cast<const uint2*>(gp + i));
                g[0] = Vec<G>::lane16(q.x, 0);
                g[1] = Vec<G>::lane16(q.x, 1);
                g[2] = Vec<G>::lane16(q.y, 0);
                g[3] = Vec<G>::lane16(q.y, 1);
            }
            if (BITS == 32) {
                m32 = *reinterpret_cast<const float4*>(static_cast<const float*>(e.m) + i);
                v32 = *reinterpret_cast<const float4*>(static_cast<const float*>(e.v) + i);
            } else {
                m8 = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(e.m) + i);
                v8 = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(e.v) + i);
            }
            return;
        }
        float wf[4], mf[4], vf[4];
        m8 = v8 = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t i = at(b, lane, j);
            const bool in = i < end;
            wf[j] = in ? e.w[i] : 0.0f;
            g[j] = in ? to_f32(gp[i]) : 0.0f;
            if (BITS == 32) {
                mf[j] = in ? static_cast<const float*>(e.m)[i] : 0.0f;
                vf[j] = in ? static_cast<const float*>(e.v)[i] : 0.0f;
            } else if (in) {
                m8 |= (uint32_t)static_cast<const uint8_t*>(e.m)[i] << (8 * j);
                v8 |= (uint32_t)static_cast<const uint8_t*>(e.v)[i] << (8 * j);
            }
        }
        w = make_float4(wf[0], wf[1], wf[2], wf[3]);
        if (BITS == 32) {
            m32 = make_float4(mf[0], mf[1], mf[2], mf[3]);
            v32 = make_float4(vf[0], vf[1], vf[2], vf[3]);
        }
    }
    __device__ __forceinline__ void step(const AdamEntry& e, const AdamConst& k, int64_t b, int64_t end, int lane)
    {
        float wf[4] = {w.x, w.y, w.z, w.w}, m[4], v[4];
        if (BITS == 32) {
            m[0] = m32.x; m[1] = m32.y; m[2] = m32.z; m[3] = m32.w;
            v[0] = v32.x; v[1] = v32.y; v[2] = v32.z; v[3] = v32.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                m[j] = moment_value<false>(m8, j, moment_base<false>(em));
                v[j] = moment_value<true>(v8, j, moment_base<true>(ev));
            }
            if (em == -128 || ev == -128) {
                // a NaN block; elements beyond the tensor's end are not to reach the maxima
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = at(b, lane, j) < end;
                    if (em == -128) m[j] = in ? __uint_as_float(0x7FC00000u) : 0.0f;
                    if (ev == -128) v[j] = in ? __uint_as_float(0x7FC00000u) : 0.0f;
                }
            }
        }
        float most_m = 0.0f, most_v = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            adam_element(k, e.decay, g[j], wf[j], m[j], v[j]);
            most_m = larger(most_m, m[j]);
            most_v = larger(most_v, v[j]);
        }
        if (BITS == 8) {
            const uint32_t tm = __reduce_max_sync(0xffffffffu, __float_as_uint(most_m));
            const uint32_t tv = __reduce_max_sync(0xffffffffu, __float_as_uint(most_v));
            em = moment_exponent<false>(tm);
            ev = moment_exponent<true>(tv);
            const uint32_t h0 = round_key(k.key + e.salt, b);
            if (tm > kMomentTop) clamp_moments(m);
            if (tv > kMomentTop) clamp_moments(v);
            uint32_t mc[4], vc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t um, uv;
                // (the low half of the element's index is below its block's end: no carry)
                round_bits(h0 + (uint32_t)(VEC ? lane * 4 + j : j * 32 + lane) * kMixIndex, um, uv);
                mc[j] = moment_code<false>(m[j], moment_base<false>(em), um);
                vc[j] = moment_code<true>(v[j], moment_base<true>(ev), uv);
            }
            m8 = mc[0] | mc[1] << 8 | mc[2] << 16 | mc[3] << 24;
            v8 = vc[0] | vc[1] << 8 | vc[2] << 16 | vc[3] << 24;
            if (em == -128) m8 = 0u;
            if (ev == -128) v8 = 0u;
            if (lane == 0) {
                e.m_exp[b / kAdamBlock] = (int8_t)em;
                e.v_exp[b / kAdamBlock] = (int8_t)ev;
            }
        }
        C* copy = static_cast<C*>(e.copy);
        if (VEC && b + kAdamBlock <= end) {
            const int64_t i = b + lane * 4;
            *reinterpret_cast<float4*>(e.w + i) = make_float4(wf[0], wf[1], wf[2], wf[3]);
            if (copy)
                *reinterpret_cast<uint2*>(copy + i) =
                    make_uint2(Vec<C>::pair16(wf[0], wf[1]), Vec<C>::pair16(wf[2], wf[3]));
            if (BITS == 32) {
                *reinterpret_cast<float4*>(static_cast<float*>(e.m) + i) = make_float4(m[0], m[1], m[2], m[3]);
                *reinterpret_cast<float4*>(static_cast<float*>(e.v) + i) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(e.m) + i) = m8;
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(e.v) + i) = v8;
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t i = at(b, lane, j);
            if (i >= end) continue;
            e.w[i] = wf[j];
            if (copy) copy[i] = from_f32<C>(wf[j]);
            if (BITS == 32) {
                static_cast<float*>(e.m)[i] = m[j];
                static_cast<float*>(e.v)[i] = v[j];
            } else {
                static_cast<uint8_t*>(e.m)[i] = (uint8_t)(m8 >> (8 * j));
                static_cast<uint8_t*>(e.v)[i] = (uint8_t)(v8 >> (8 * j));
            }
        }
    }
};

// A warp takes UNROLL blocks of 128 elements at a time, all their loads before the first step.
template <typename G, typename C, int BITS, bool VEC, int UNROLL>
__device__ __forceinline__ void adam_chunk(const AdamEntry& e, const AdamConst& k, int64_t base, int64_t end)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int64_t kStep = (kAdamThreads / 32) * kAdamBlock;
    for (int64_t b = base + warp * kAdamBlock; b < end; b += UNROLL * kStep) {
        AdamPiece<G, C, BITS, VEC> p[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
            if (b + u * kStep < end) p[u].load(e, b + u * kStep, end, lane);
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
            if (b + u * kStep < end) p[u].step(e, k, b + u * kStep, end, lane);
    }
}

template <typename G, typename C, int BITS>
__global__ void __launch_bounds__(kAdamThreads) k_adamw(const __grid_constant__ AdamTable tab, const AdamConst k)
{
    griddep_wait();
    griddep_launch_dependents();
    const AdamEntry& e = tab.e[find_entry(tab, blockIdx.x)];
    const int64_t base = e.from + (int64_t)(blockIdx.x - e.first_chunk) * kAdamChunk;
    const int64_t end = min(e.n, base + kAdamChunk);
    if (e.vec) adam_chunk<G, C, BITS, true, 2>(e, k, base, end);
    else adam_chunk<G, C, BITS, false, 1>(e, k, base, end);
}

// ------------------------------------------------------ whole chunks, 8-bit moments
//
// The step reads 8 and writes 8 bytes an element (bf16 gradients and copies), with about 105
// instructions between, and their issue bounds it (138M weights: 480 us, 332 at the memory's rate;
// roots and quotients take 7 % of it, the rounding's hash 9 %), so loads may not wait for
// arithmetic. A producer thread keeps a ring of chunks of 2048 elements coming into shared
// memory by bulk copies, and three teams of eight warps take them in turn, half a warp to a
// block of 128 elements, eight elements to a lane. Chunks whose arrays start on 16-byte boundaries come here;
// the rest (a tensor's last part, odd places) takes k_adamw.
constexpr int kRingChunk = 2048;
constexpr int kRingTensor = 32 * kRingChunk;     // elements of a tensor from which it goes this way
constexpr int kRingWarps = 8, kRingTeams = 3;
constexpr int kRingThreads = (kRingTeams * kRingWarps + 1) * 32;

template <typename G>
struct RingCfg {
    static constexpr int G_AT = kRingChunk * 4, M_AT = G_AT + kRingChunk * (int)sizeof(G), V_AT = M_AT + kRingChunk;
    static constexpr int BYTES = V_AT + kRingChunk;
    static constexpr int STAGES = 200 * 1024 / BYTES;
};

template <typename G, typename C>
__global__ void __launch_bounds__(kRingThreads, 1)
    k_adamw_ring(const __grid_constant__ AdamTable tab, const AdamConst k, uint32_t chunks, int* __restrict__ err)
{
    using Cfg = RingCfg<G>;
    constexpr int STAGES = Cfg::STAGES;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint64_t full[STAGES], empty[STAGES];
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kRingWarps);
        }
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    int stage = 0;
    uint32_t phase = 0;
    if (warp == kRingTeams * kRingWarps) {
        if (lane) return;
        int entry = 0;
        for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
            entry = next_entry(tab, entry, c);
            const AdamEntry& e = tab.e[entry];
            const int64_t base = (int64_t)(c - e.first_chunk) * kRingChunk;
            if (!mbar_wait(&empty[stage], phase ^ 1, &abort_flag, err)) break;
            uint8_t* p = smem + stage * Cfg::BYTES;
            mbar_arrive_expect_tx(&full[stage], Cfg::BYTES);
            bulk_load(p, e.w + base, kRingChunk * 4, &full[stage]);
            bulk_load(p + Cfg::G_AT, static_cast<const G*>(e.g) + base, kRingChunk * sizeof(G), &full[stage]);
            bulk_load(p + Cfg::M_AT, static_cast<const uint8_t*>(e.m) + base, kRingChunk, &full[stage]);
            bulk_load(p + Cfg::V_AT, static_cast<const uint8_t*>(e.v) + base, kRingChunk, &full[stage]);
            if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
        // (the teams may have given up: the block stays until every copy has landed)
        ring_landed(full, STAGES, RingPlace{stage, phase}.lap_before(), STAGES);
        return;
    }
    const int team = warp / kRingWarps, half = lane >> 4, hl = lane & 15;
    const int block = warp % kRingWarps * 2 + half, at = block * kAdamBlock + hl * 4;     // and at + 64
    const uint32_t stride = kRingTeams * gridDim.x;
    uint32_t c = blockIdx.x + team * gridDim.x;
    stage = team;
    int em = 0, ev = 0;                  // the next chunk's exponents come one chunk ahead
    int entry = 0;
    if (c < chunks) {
        entry = find_entry(tab, c);
        const AdamEntry& e = tab.e[entry];
        const int64_t b = (int64_t)(c - e.first_chunk) * (kRingChunk / kAdamBlock) + block;
        em = e.m_exp[b];
        ev = e.v_exp[b];
    }
    for (; c < chunks; c += stride) {
        const AdamEntry& e = tab.e[entry];
        const int64_t base = (int64_t)(c - e.first_chunk) * kRingChunk;
        int em_next = 0, ev_next = 0;
        if (c + stride < chunks) {
            entry = next_entry(tab, entry, c + stride);
            const AdamEntry& n = tab.e[entry];
            const int64_t b = (int64_t)(c + stride - n.first_chunk) * (kRingChunk / kAdamBlock) + block;
            em_next = n.m_exp[b];
            ev_next = n.v_exp[b];
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, &abort_flag, err))) return;
        const uint8_t* p = smem + stage * Cfg::BYTES;
        float w[8], g[8], m[8], v[8];
        uint32_t mc[2], vc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = at + 64 * h;
            const float4 q = *reinterpret_cast<const float4*>(p + i * 4);
            w[4 * h] = q.x; w[4 * h + 1] = q.y; w[4 * h + 2] = q.z; w[4 * h + 3] = q.w;
            if constexpr (sizeof(G) == 4) {
                const float4 r = *reinterpret_cast<const float4*>(p + Cfg::G_AT + i * 4);
                g[4 * h] = r.x; g[4 * h + 1] = r.y; g[4 * h + 2] = r.z; g[4 * h + 3] = r.w;
            } else {
                const uint2 r = *reinterpret_cast<const uint2*>(p + Cfg::G_AT + i * 2);
                g[4 * h] = Vec<G>::lane16(r.x, 0);
                g[4 * h + 1] = Vec<G>::lane16(r.x, 1);
                g[4 * h + 2] = Vec<G>::lane16(r.y, 0);
                g[4 * h + 3] = Vec<G>::lane16(r.y, 1);
            }
            mc[h] = *reinterpret_cast<const uint32_t*>(p + Cfg::M_AT + i);
            vc[h] = *reinterpret_cast<const uint32_t*>(p + Cfg::V_AT + i);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        stage += kRingTeams;
        if (stage >= STAGES) { stage -= STAGES; phase ^= 1; }
        const uint32_t base_m = moment_base<false>(em), base_v = moment_base<true>(ev);
        float most_m = 0.0f, most_v = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m[j] = moment_value<false>(mc[j >> 2], j & 3, base_m);
            v[j] = moment_value<true>(vc[j >> 2], j & 3, base_v);
        }
        if (em == -128 || ev == -128)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (em == -128) m[j] = __uint_as_float(0x7FC00000u);
                if (ev == -128) v[j] = __uint_as_float(0x7FC00000u);
            }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            adam_element(k, e.decay, g[j], w[j], m[j], v[j]);
            most_m = larger(most_m, m[j]);
            most_v = larger(most_v, v[j]);
        }
        uint32_t tm = __float_as_uint(most_m), tv = __float_as_uint(most_v);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            tm = max(tm, __shfl_xor_sync(0xffffffffu, tm, o));
            tv = max(tv, __shfl_xor_sync(0xffffffffu, tv, o));
        }
        em = moment_exponent<false>(tm);
        ev = moment_exponent<true>(tv);
        if (tm > kMomentTop) clamp_moments(m);
        if (tv > kMomentTop) clamp_moments(v);
        const uint32_t to_m = moment_base<false>(em), to_v = moment_base<true>(ev);
        const uint32_t h0 = round_key(k.key + e.salt, base + at);
        C* copy = static_cast<C*>(e.copy);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t cm[4], cv[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t um, uv;
                // (chunks do not straddle a multiple of 2^32: no carry)
                round_bits(h0 + (uint32_t)(64 * h + j) * kMixIndex, um, uv);
                cm[j] = moment_code<false>(m[4 * h + j], to_m, um);
                cv[j] = moment_code<true>(v[4 * h + j], to_v, uv);
            }
            uint32_t m8 = __byte_perm(__byte_perm(cm[0], cm[1], 0x0040), __byte_perm(cm[2], cm[3], 0x0040), 0x5410);
            uint32_t v8 = __byte_perm(__byte_perm(cv[0], cv[1], 0x0040), __byte_perm(cv[2], cv[3], 0x0040), 0x5410);
            if (em == -128) m8 = 0u;
            if (ev == -128) v8 = 0u;
            const int64_t i = base + at + 64 * h;
            *reinterpret_cast<float4*>(e.w + i) = make_float4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
            if (copy)
                *reinterpret_cast<uint2*>(copy + i) = make_uint2(Vec<C>::pair16(w[4 * h], w[4 * h + 1]),
                                                                 Vec<C>::pair16(w[4 * h + 2], w[4 * h + 3]));
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(e.m) + i) = m8;
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(e.v) + i) = v8;
        }
        if (hl == 0) {
            const int64_t b = base / kAdamBlock + block;
            e.m_exp[b] = (int8_t)em;
            e.v_exp[b] = (int8_t)ev;
        }
        em = em_next;
        ev = ev_next;
    }
}

template <bool SECOND>
__device__ __forceinline__ float moment_or_nan(uint32_t codes, int j, int e)
{
    return e == -128 ? __uint_as_float(0x7FC00000u) : moment_value<SECOND>(codes, j, moment_base<SECOND>(e));
}

// The values of 8-bit moments, the tensors one after another in m_out and v_out.
struct MomentEntry {
    const uint8_t* m;
    const uint8_t* v;
    const int8_t* m_exp;
    const int8_t* v_exp;
    int64_t n, out;         // first element of this tensor's values
    uint32_t first_chunk;
    int32_t vec;            // four elements at a time
};
constexpr int kMomentEntries = 64;
struct MomentTable {
    int32_t n;
    MomentEntry e[kMomentEntries];
};

__device__ __forceinline__ void store_four(float* p, const float (&v)[4])
{
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_four(__nv_bfloat16* p, const float (&v)[4])
{
    *reinterpret_cast<uint2*>(p) =
        make_uint2(Vec<__nv_bfloat16>::pair16(v[0], v[1]), Vec<__nv_bfloat16>::pair16(v[2], v[3]));
}

template <typename O>
__global__ void __launch_bounds__(kAdamThreads)
    k_moments(const __grid_constant__ MomentTable tab, O* __restrict__ m_out, O* __restrict__ v_out)
{
    griddep_wait();
    griddep_launch_dependents();
    int lo = 0, hi = tab.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.e[mid].first_chunk <= blockIdx.x) lo = mid; else hi = mid - 1;
    }
    const MomentEntry& e = tab.e[lo];
    const int64_t base = (int64_t)(blockIdx.x - e.first_chunk) * kAdamChunk;
    const int64_t end = min(e.n, base + kAdamChunk);
    if (e.vec) {
        for (int64_t i = base + threadIdx.x * 4; i < end; i += kAdamThreads * 4) {
            const uint32_t m = *reinterpret_cast<const uint32_t*>(e.m + i), v = *reinterpret_cast<const uint32_t*>(e.v + i);
            const int em = e.m_exp[i / kAdamBlock], ev = e.v_exp[i / kAdamBlock];
            float mf[4], vf[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mf[j] = moment_or_nan<false>(m, j, em);
                vf[j] = moment_or_nan<true>(v, j, ev);
            }
            if (m_out) store_four(m_out + e.out + i, mf);
            if (v_out) store_four(v_out + e.out + i, vf);
        }
        return;
    }
    for (int64_t i = base + threadIdx.x; i < end; i += kAdamThreads) {
        if (m_out) m_out[e.out + i] = from_f32<O>(moment_or_nan<false>(e.m[i], 0, e.m_exp[i / kAdamBlock]));
        if (v_out) v_out[e.out + i] = from_f32<O>(moment_or_nan<true>(e.v[i], 0, e.v_exp[i / kAdamBlock]));
    }
}

// ------------------------------------------------------------------- launchers

template <typename G, typename C>
static int launch_ring(const AdamTable& t, const AdamConst& k, uint32_t chunks, cudaStream_t s)
{
    constexpr int kBytes = RingCfg<G>::STAGES * RingCfg<G>::BYTES;
    if (cudaFuncSetAttribute(k_adamw_ring<G, C>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) != cudaSuccess)
        return set_error(ITO_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(cudaGetLastError()));
    int* err = device_error_word();
    if (!err) return set_error(ITO_ERR_CUDA, "device error word unavailable");
    launch_pdl(k_adamw_ring<G, C>, std::min<uint32_t>(chunks, num_sms()), kRingThreads, kBytes, s, t, k, chunks, err);
    return launch_status("adamw");
}

// ring: whole chunks of 8-bit states
template <typename G, typename C>
static int launch_adamw(const AdamTable& t, const AdamConst& k, int bits, bool ring, uint32_t chunks, cudaStream_t s)
{
    if (ring) return launch_ring<G, C>(t, k, chunks, s);
    if (bits == 8) launch_pdl(k_adamw<G, C, 8>, chunks, kAdamThreads, 0, s, t, k);
    else launch_pdl(k_adamw<G, C, 32>, chunks, kAdamThreads, 0, s, t, k);
    return launch_status("adamw");
}

template <typename G>
static int launch_adamw(const AdamTable& t, const AdamConst& k, int bits, bool ring, int copy_type, uint32_t chunks,
                        cudaStream_t s)
{
    if (copy_type == ITO_F16) return launch_adamw<G, __half>(t, k, bits, ring, chunks, s);
    return launch_adamw<G, __nv_bfloat16>(t, k, bits, ring, chunks, s);
}

// The parts of the tensors that one kernel takes, in launches of up to kAdamEntries tensors: the
// whole chunks of `whole` tensors (ring), or what that leaves.
static int run_adamw(const ito_adamw_tensor* tensors, int n_tensors, const ito_adamw_params* p, const AdamConst& k,
                     bool ring, int64_t ring_from, cudaStream_t s)
{
    const size_t g_size = type_bytes(p->grad_type);
    AdamTable tab;
    for (int i = 0; i < n_tensors;) {
        tab.n = 0;
        uint64_t chunks = 0;
        for (; i < n_tensors && tab.n < kAdamEntries; ++i) {
            const ito_adamw_tensor& a = tensors[i];
            const bool aligned = aligned_to(a.w, 16) && aligned_to(a.g, 16) && aligned_to(a.m, 16) &&
                                 aligned_to(a.v, 16) && aligned_to(a.copy, 8);
            // elements that the ring takes of this tensor
            const int64_t whole = ring_from && aligned && a.n >= ring_from ? a.n / kRingChunk * kRingChunk : 0;
            const int64_t from = ring ? 0 : whole, n = ring ? whole : a.n;
            const uint64_t c = ring ? (uint64_t)(n / kRingChunk) : (uint64_t)(n - from + kAdamChunk - 1) / kAdamChunk;
            if (chunks + c > 0x7fffffffu) break;
            if (!c) continue;
            const size_t state = p->state_bits == 32 ? 16 : 4;
            const int vec = aligned_to(a.w, 16) && aligned_to(a.g, 4 * g_size) && aligned_to(a.copy, 8) &&
                            aligned_to(a.m, state) && aligned_to(a.v, state);
            AdamEntry& e = tab.e[tab.n++];
            e = AdamEntry{a.w, a.g, a.copy, a.m, a.v, a.m_exp, a.v_exp, n, from, (uint32_t)chunks,
                          (float)(1.0 - p->lr * a.weight_decay), vec, (uint32_t)i * 0x510E527Fu};
            chunks += c;
        }
        if (!chunks) continue;
        int r;
        if (p->grad_type == ITO_F32) r = launch_adamw<float>(tab, k, p->state_bits, ring, p->copy_type, (uint32_t)chunks, s);
        else if (p->grad_type == ITO_BF16)
            r = launch_adamw<__nv_bfloat16>(tab, k, p->state_bits, ring, p->copy_type, (uint32_t)chunks, s);
        else r = launch_adamw<__half>(tab, k, p->state_bits, ring, p->copy_type, (uint32_t)chunks, s);
        if (r) return r;
    }
    return ITO_OK;
}

static int check_tensor(const ito_adamw_tensor& a, int i, int bits)
{
    if (a.n < 0 || a.n > (int64_t(1) << 40)) return set_error(ITO_ERR_SHAPE, "tensor %d: n outside 0 .. 2^40", i);
    if (a.n == 0) return ITO_OK;
    if (!a.m || !a.v) return set_error(ITO_ERR_ARG, "tensor %d: NULL state pointer", i);
    if (bits == 8 && (!a.m_exp || !a.v_exp)) return set_error(ITO_ERR_ARG, "tensor %d: NULL exponent pointer", i);
    if (bits == 32 && (!aligned_to(a.m, 4) || !aligned_to(a.v, 4)))
        return set_error(ITO_ERR_ARG, "tensor %d: misaligned state pointer", i);
    return ITO_OK;
}

}  // namespace ito

using namespace ito;

extern "C" {

int ito_adamw_step(const ito_adamw_tensor* tensors, int n_tensors, const ito_adamw_params* p, void* stream)
{
    if (!tensors || !p) return set_error(ITO_ERR_ARG, "NULL argument");
    if (n_tensors < 1) return set_error(ITO_ERR_SHAPE, "n_tensors must be >= 1");
    if (p->state_bits != 32 && p->state_bits != 8) return set_error(ITO_ERR_ARG, "state_bits must be 32 or 8");
    if (!type_known(p->grad_type)) return set_error(ITO_ERR_ARG, "unknown grad_type");
    if (p->copy_type != ITO_BF16 && p->copy_type != ITO_F16)
        return set_error(ITO_ERR_ARG, "copy_type must be ITO_BF16 or ITO_F16");
    if (p->step < 1) return set_error(ITO_ERR_ARG, "step must be >= 1");
    if (!(p->beta1 >= 0 && p->beta1 < 1) || !(p->beta2 >= 0 && p->beta2 < 1))
        return set_error(ITO_ERR_ARG, "betas must be in [0, 1)");
    if (!(p->eps >= 0)) return set_error(ITO_ERR_ARG, "eps must be >= 0");
    for (int i = 0; i < n_tensors; ++i) {
        const ito_adamw_tensor& a = tensors[i];
        const int r = check_tensor(a, i, p->state_bits);
        if (r) return r;
        if (a.n == 0) continue;
        if (!a.w || !a.g) return set_error(ITO_ERR_ARG, "tensor %d: NULL weight or gradient pointer", i);
        if (!aligned_to(a.w, 4) || !aligned_to(a.g, type_bytes(p->grad_type)) || !aligned_to(a.copy, 2))
            return set_error(ITO_ERR_ARG, "tensor %d: misaligned pointer", i);
    }
    AdamConst k;
    const double t = (double)p->step;
    k.b1 = (float)p->beta1;
    k.c1 = (float)(1.0 - p->beta1);
    k.b2 = (float)p->beta2;
    k.c2 = (float)(1.0 - p->beta2);
    k.eps = (float)p->eps;
    k.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(p->beta2, t)));
    k.alpha = (float)(p->lr / (1.0 - std::pow(p->beta1, t)));
    k.grad_scale = (float)p->grad_scale;
    k.key = p->seed + (uint32_t)(uint64_t)p->step * 0x9E3779B1u;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    // the ring pays for tensors of many chunks, where all of them together keep it full
    int64_t total = 0;
    for (int i = 0; i < n_tensors; ++i)
        if (tensors[i].n >= kRingTensor) total += tensors[i].n;
    const int64_t ring_from = p->state_bits == 8 && total >= (int64_t)8 * kRingChunk * num_sms() ? kRingTensor : 0;
    if (ring_from) {
        const int r = run_adamw(tensors, n_tensors, p, k, true, ring_from, s);
        if (r) return r;
    }
    return run_adamw(tensors, n_tensors, p, k, false, ring_from, s);
}

int ito_adamw_moments(const ito_adamw_tensor* tensors, int n_tensors, int out_type, void* m_out, void* v_out,
                      void* stream)
{
    if (!tensors || (!m_out && !v_out)) return set_error(ITO_ERR_ARG, "NULL argument");
    if (n_tensors < 1) return set_error(ITO_ERR_SHAPE, "n_tensors must be >= 1");
    if (out_type != ITO_F32 && out_type != ITO_BF16)
        return set_error(ITO_ERR_ARG, "out_type must be ITO_F32 or ITO_BF16");
    if (!aligned_to(m_out, type_bytes(out_type)) || !aligned_to(v_out, type_bytes(out_type)))
        return set_error(ITO_ERR_ARG, "misaligned output pointer");
    for (int i = 0; i < n_tensors; ++i) {
        const int r = check_tensor(tensors[i], i, 8);
        if (r) return r;
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    MomentTable tab;
    int64_t out = 0;
    for (int i = 0; i < n_tensors;) {
        tab.n = 0;
        uint64_t chunks = 0;
        for (; i < n_tensors && tab.n < kMomentEntries; ++i) {
            const ito_adamw_tensor& a = tensors[i];
            const uint64_t c = ((uint64_t)a.n + kAdamChunk - 1) / kAdamChunk;
            if (chunks + c > 0x7fffffffu) break;
            if (!c) continue;
            const int64_t at = out * (int64_t)type_bytes(out_type);
            const int vec = a.n % 4 == 0 && aligned_to(a.m, 4) && aligned_to(a.v, 4) && at % 16 == 0 &&
                            aligned_to(m_out, 16) && aligned_to(v_out, 16);
            tab.e[tab.n++] = MomentEntry{static_cast<const uint8_t*>(a.m), static_cast<const uint8_t*>(a.v), a.m_exp,
                                         a.v_exp, a.n, out, (uint32_t)chunks, vec};
            chunks += c;
            out += a.n;
        }
        if (!chunks) continue;
        if (out_type == ITO_F32)
            launch_pdl(k_moments<float>, (uint32_t)chunks, kAdamThreads, 0, s, tab, static_cast<float*>(m_out),
                       static_cast<float*>(v_out));
        else
            launch_pdl(k_moments<__nv_bfloat16>, (uint32_t)chunks, kAdamThreads, 0, s, tab,
                       static_cast<__nv_bfloat16*>(m_out), static_cast<__nv_bfloat16*>(v_out));
        const int r = launch_status("moments");
        if (r) return r;
    }
    return ITO_OK;
}

}  // extern "C"
