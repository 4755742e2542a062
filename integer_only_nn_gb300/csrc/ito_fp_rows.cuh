// A few rows of x times one or two weights, with the ends that such calls take.
#pragma once

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

// warps of a block, at most
template <FpEnd END, int NT>
constexpr int kRowsWarps = END == FpEnd::Linear || NT > 2 ? 8 : 16;
// These products too cut off what a sum's 24 bits cannot hold at each step of 16 k, and a warp's chain of them grows
// with IC (16384 in 4 warps: a logit of positive products short by 1.3e-5 of itself). So a logit's chains end every 1024 k
// of a warp, and their sums are added up, rounded. (The linear and the gated layer's results are rounded to 16 bits.)
constexpr int kRowsChain = 1024;
// steps of 32 k whose loads of W are in flight together
template <FpEnd END>
constexpr int kRowsSteps = END == FpEnd::Linear ? 4 : 2;

// VEC: both operands' rows start on 16-byte boundaries and IC is a multiple of 8. Of other rows each eight
// elements come in words and a shift (Eight16; the plain linear layer, whose sums keep their
// order and so their four steps, loads them one by one). The gated layer
// streams two weights, 16 rows of each to a block, half as many steps of each ahead (the same bytes
// in flight and registers). LONG: logits of rows that take a warp more than one chain; the sums wait in shared
// memory, because registers for them cost blocks of an SM (13 x 1531 x 50001 f16 143 us instead of 122). A Loss leaves each
// row's parts of 16 columns; DLogits are as from the tensor cores' kernels.
template <FpEnd END, int NT, bool VEC, bool LONG>
__global__ void __launch_bounds__(kRowsWarps<END, NT> * 32)
    k_fp_rows(const uint16_t* __restrict__ x, int64_t ldx, const uint16_t* __restrict__ W, int64_t ldw,
              const uint16_t* __restrict__ W2, int64_t ldw2, int B, int IC, int OC, const __grid_constant__ FpEpilogue e,
              const __grid_constant__ FpMore more, int* err)
{
    constexpr int U = kRowsSteps<END>, WS = END == FpEnd::Gated ? 2 : 1;
    constexpr bool SHIFT = !VEC && END != FpEnd::Linear;
    using Raw = typename std::conditional<SHIFT, Eight16, uint4>::type;
    extern __shared__ float rows_part[];
    float(*const part)[WS][16 * 8 * NT] = reinterpret_cast<float(*)[WS][16 * 8 * NT]>(rows_part);
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int warps = blockDim.x >> 5;
    const int oc0 = blockIdx.x * 16;
    const bool in0 = oc0 + g < OC, in1 = oc0 + g + 8 < OC;
    const uint16_t *w0[WS], *w1[WS];
    w0[0] = W + (int64_t)(in0 ? oc0 + g : 0) * ldw;
    w1[0] = W + (int64_t)(in1 ? oc0 + g + 8 : 0) * ldw;
    if (WS == 2) {
        w0[WS - 1] = W2 + (int64_t)(in0 ? oc0 + g : 0) * ldw2;
        w1[WS - 1] = W2 + (int64_t)(in1 ? oc0 + g + 8 : 0) * ldw2;
    }
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const uint16_t* const w_end[2] = {W + (OC - 1) * ldw + IC, WS == 2 ? W2 + (OC - 1) * ldw2 + IC : nullptr};
    // only a weight's first and last row have words that reach beyond it
    const bool inner0 = oc0 + g > 0 && oc0 + g + 1 < OC, inner1 = oc0 + g + 9 < OC;
    auto load = [&](const uint16_t* row, int k, bool in, bool inner, int h) -> Raw {
        if constexpr (SHIFT) {
            Raw e;
            e.w[0] = e.w[1] = e.w[2] = e.w[3] = e.w[4] = 0u;
            if (in && k + 8 <= IC && (inner || Eight16::whole(row + k, h ? W2 : W, w_end[h]))) e.load(row + k);
            return e;
        } else if constexpr (VEC) {
            return in && k < IC ? load_once(row + k) : zero;
        } else {
            return in && k < IC ? load_eight(row, k, IC, false) : zero;
        }
    };
    // what was loaded, as the eight elements (those at a row's or the weight's end are loaded here)
    auto eight = [&](const Raw& e, const uint16_t* row, int k, bool in, bool inner, int h) -> uint4 {
        if constexpr (SHIFT) {
            if (!in || k >= IC) return zero;
            if (k + 8 <= IC && (inner || Eight16::whole(row + k, h ? W2 : W, w_end[h]))) return e.get(row + k);
            return load_eight(row, k, IC, false);
        } else {
            return e;
        }
    };
    const uint16_t* const x_end = x + (B - 1) * ldx + IC;
    auto load_x = [&](const uint16_t* row, int k, bool in) -> uint4 {
        if (!in || k >= IC) return zero;
        if constexpr (SHIFT) {
            if (k + 8 <= IC && Eight16::whole(row + k, x, x_end)) {
                Eight16 e;
                e.load(row + k);
                return e.get(row + k);
            }
        }
        return load_eight(row, k, IC, VEC);
    };
    float c[WS][NT][4];
    auto clear = [&] {
#pragma unroll
        for (int h = 0; h < WS; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) c[h][n][i] = 0.0f;
    };
    clear();
    // this warp's sums, put down or added to what it has put down
    auto put = [&](bool again) {
#pragma unroll
        for (int h = 0; h < WS; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float& at = part[warp][h][(n * 8 + 2 * t + (i & 1)) * 16 + g + 8 * (i >> 1)];
                    at = again ? at + c[h][n][i] : c[h][n][i];
                }
    };
    Raw a[WS][U], b[WS][U];
    const int stride = warps * U * 32;
    int k0 = warp * U * 32, steps = 0;               // (steps of the chain)
    bool again = false;
#pragma unroll
    for (int h = 0; h < WS; ++h)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[h][u] = load(w0[h], k0 + u * 32 + t * 8, in0, inner0, h);
            b[h][u] = load(w1[h], k0 + u * 32 + t * 8, in1, inner1, h);
        }
    for (; k0 < IC; k0 += stride) {
        // the next steps' rows of W are on their way while these are multiplied
        Raw an[WS][U], bn[WS][U];
#pragma unroll
        for (int h = 0; h < WS; ++h)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                an[h][u] = load(w0[h], k0 + stride + u * 32 + t * 8, in0, inner0, h);
                bn[h][u] = load(w1[h], k0 + stride + u * 32 + t * 8, in1, inner1, h);
            }
        uint4 wa[WS][U], wb[WS][U];
#pragma unroll
        for (int h = 0; h < WS; ++h)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                wa[h][u] = eight(a[h][u], w0[h], k0 + u * 32 + t * 8, in0, inner0, h);
                wb[h][u] = eight(b[h][u], w1[h], k0 + u * 32 + t * 8, in1, inner1, h);
            }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool in = n * 8 + g < B;
            const uint16_t* xr = x + (int64_t)(in ? n * 8 + g : 0) * ldx;
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * 32 + t * 8;
                v[u] = load_x(xr, k, in);
            }
#pragma unroll
            for (int h = 0; h < WS; ++h)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    mma_16816(e.type, c[h][n], wa[h][u].x, wb[h][u].x, wa[h][u].y, wb[h][u].y, v[u].x, v[u].y);
                    mma_16816(e.type, c[h][n], wa[h][u].z, wb[h][u].z, wa[h][u].w, wb[h][u].w, v[u].z, v[u].w);
                }
        }
#pragma unroll
        for (int h = 0; h < WS; ++h)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                a[h][u] = an[h][u];
                b[h][u] = bn[h][u];
            }
        if (LONG && ++steps == kRowsChain / (U * 32)) {
            put(again);
            clear();
            again = true;
            steps = 0;
        }
    }
    put(LONG && again);
    __syncthreads();
    // (whole warps go round: 16 x 8 NT sums and the block's threads are multiples of 32)
    for (int i = threadIdx.x; i < 16 * 8 * NT; i += blockDim.x) {
        const int row = i >> 4, oc = oc0 + (i & 15);
        const bool in = row < B && oc < OC;
        float s[WS];
#pragma unroll
        for (int h = 0; h < WS; ++h) {
            s[h] = part[0][h][i];
            for (int w = 1; w < warps; ++w) s[h] += part[w][h][i];
        }
        if (END == FpEnd::Loss) {
            if (in && oc == more.targets[row]) more.hit[row] = s[0];
            float m = oc < OC ? s[0] : -INFINITY, sum = oc < OC ? 1.0f : 0.0f;
            fp_softmax_warp(m, sum, 16);
            if (row < B && (i & 15) == 0) more.part[(int64_t)blockIdx.x * B + row] = make_float2(m, sum);
        } else if (in) {
            if (END == FpEnd::DLogits) {
                SlopeRow slope;
                slope.load(more, B, row, oc == 0 && more.first == 0, err);
                store_typed(e.y, e.type, row * e.ldy + oc, slope.at(s[0], oc));
            } else if (END == FpEnd::Gated) fp_finish_gated(e, more, row, oc, s[0], s[WS - 1]);
            else fp_finish(e, row, oc, s[0]);
        }
    }
}

template <FpEnd END, int NT>
static int fp_launch_rows(const void* x, int64_t ldx, const void* W, int64_t ldw, const void* W2, int64_t ldw2, int B,
                          int IC, int OC, const FpEpilogue& e, const FpMore& more, cudaStream_t s)
{
    int* const err = END == FpEnd::DLogits ? device_error_word() : nullptr;
    if (END == FpEnd::DLogits && !err) return set_error(ITO_ERR_CUDA, "device error word unavailable");
    const bool vec = fp_rows_vec(x, ldx, W, ldw, B, IC, OC) && (!W2 || fp_tma_rows(W2, ldw2, OC, IC));
    // With blocks for two to an SM and more, 4 warps each let all of them run at the same time (one row of 4096 ->
    // 8192: 22 us instead of 25, of 4096 -> 131072 classes 162 instead of 173); fewer blocks have more warps. (The
    // number of warps is part of the sums' order: the plain linear layer keeps its.)
    const int blocks = (OC + 15) / 16;
    const int most = END == FpEnd::Linear ? 8 : std::min(kRowsWarps<END, NT>, blocks < num_sms() ? 16 : blocks < 2 * num_sms() ? 8 : 4);
    constexpr int step = 32 * kRowsSteps<END>;
    const int warps = std::min(most, std::max(1, (IC + step - 1) / step));
    // (more than 16 rows at any alignment: the plain linear layer alone, see fp_few_rows; others have one instance. More
    // than 16 rows of logits are no longer than a chain of 8 warps, see fp_few_logits)
    constexpr bool LOGITS = (END == FpEnd::Loss || END == FpEnd::DLogits) && NT <= 2, ANY = END == FpEnd::Linear || NT <= 2;
    if (!ANY && !vec) return set_error(ITO_ERR_ARG, "rows that do not start on 16-byte boundaries");
    const bool lengthy = LOGITS && IC > warps * kRowsChain;
    auto* kern = lengthy ? k_fp_rows<END, NT, true, LOGITS> : k_fp_rows<END, NT, true, false>;
    if (!vec) kern = lengthy ? k_fp_rows<END, NT, !ANY, LOGITS> : k_fp_rows<END, NT, !ANY, false>;
    launch_pdl(kern, (OC + 15) / 16, warps * 32,
               (size_t)warps * (END == FpEnd::Gated ? 2 : 1) * 16 * 8 * NT * sizeof(float), s,
               static_cast<const uint16_t*>(x), ldx, static_cast<const uint16_t*>(W), ldw,
               static_cast<const uint16_t*>(W2), ldw2, B, IC, OC, e, more, err);
    return launch_status("linear");
}

template <FpEnd END>
static int fp_run_rows(const void* x, int64_t ldx, const void* W, int64_t ldw, const void* W2, int64_t ldw2, int B, int IC,
                       int OC, const FpEpilogue& e, const FpMore& more, cudaStream_t s)
{
    if (B <= 8) return fp_launch_rows<END, 1>(x, ldx, W, ldw, W2, ldw2, B, IC, OC, e, more, s);
    if (B <= 16) return fp_launch_rows<END, 2>(x, ldx, W, ldw, W2, ldw2, B, IC, OC, e, more, s);
    if (B <= 24) return fp_launch_rows<END, 3>(x, ldx, W, ldw, W2, ldw2, B, IC, OC, e, more, s);
    return fp_launch_rows<END, 4>(x, ldx, W, ldw, W2, ldw2, B, IC, OC, e, more, s);
}

}  // namespace ito
