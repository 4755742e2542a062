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

constexpr int kRowsWarps = 8;        // of a block, at most
// steps of 32 k whose loads of W are in flight together
template <FpEnd END>
constexpr int kRowsSteps = END == FpEnd::Gated ? 2 : 4;

// VEC: both operands' rows start on 16-byte boundaries and IC is a multiple of 8. The gated layer
// streams two weights, 16 rows of each to a block, half as many steps of each ahead (the same bytes
// in flight and registers). A Loss leaves each row's parts of 16 columns.
template <FpEnd END, int NT, bool VEC>
__global__ void __launch_bounds__(kRowsWarps * 32)
    k_fp_rows(const uint16_t* __restrict__ x, int64_t ldx, const uint16_t* __restrict__ W, int64_t ldw,
              const uint16_t* __restrict__ W2, int64_t ldw2, int B, int IC, int OC, const __grid_constant__ FpEpilogue e,
              const __grid_constant__ FpMore more)
{
    constexpr int U = kRowsSteps<END>, WS = END == FpEnd::Gated ? 2 : 1;
    __shared__ float part[kRowsWarps][WS][16 * 8 * NT];
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
    auto load = [&](const uint16_t* row, int k, bool in) {
        if (VEC) return in && k < IC ? load_once(row + k) : zero;
        return in && k < IC ? load_eight(row, k, IC, false) : zero;
    };
    float c[WS][NT][4];
#pragma unroll
    for (int h = 0; h < WS; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) c[h][n][i] = 0.0f;
    uint4 a[WS][U], b[WS][U];
    const int stride = warps * U * 32;
    int k0 = warp * U * 32;
#pragma unroll
    for (int h = 0; h < WS; ++h)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[h][u] = load(w0[h], k0 + u * 32 + t * 8, in0);
            b[h][u] = load(w1[h], k0 + u * 32 + t * 8, in1);
        }
    for (; k0 < IC; k0 += stride) {
        // the next steps' rows of W are on their way while these are multiplied
        uint4 an[WS][U], bn[WS][U];
#pragma unroll
        for (int h = 0; h < WS; ++h)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                an[h][u] = load(w0[h], k0 + stride + u * 32 + t * 8, in0);
                bn[h][u] = load(w1[h], k0 + stride + u * 32 + t * 8, in1);
            }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool in = n * 8 + g < B;
            const uint16_t* xr = x + (int64_t)(in ? n * 8 + g : 0) * ldx;
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * 32 + t * 8;
                v[u] = in && k < IC ? load_eight(xr, k, IC, VEC) : zero;
            }
#pragma unroll
            for (int h = 0; h < WS; ++h)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    mma_16816(e.type, c[h][n], a[h][u].x, b[h][u].x, a[h][u].y, b[h][u].y, v[u].x, v[u].y);
                    mma_16816(e.type, c[h][n], a[h][u].z, b[h][u].z, a[h][u].w, b[h][u].w, v[u].z, v[u].w);
                }
        }
#pragma unroll
        for (int h = 0; h < WS; ++h)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                a[h][u] = an[h][u];
                b[h][u] = bn[h][u];
            }
    }
#pragma unroll
    for (int h = 0; h < WS; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[warp][h][(n * 8 + 2 * t + (i & 1)) * 16 + g + 8 * (i >> 1)] = c[h][n][i];
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
            if (END == FpEnd::Gated) fp_finish_gated(e, more, row, oc, s[0], s[WS - 1]);
            else fp_finish(e, row, oc, s[0]);
        }
    }
}

template <FpEnd END, int NT>
static int fp_launch_rows(const void* x, int64_t ldx, const void* W, int64_t ldw, const void* W2, int64_t ldw2, int B,
                          int IC, int OC, const FpEpilogue& e, const FpMore& more, cudaStream_t s)
{
    constexpr int STEP = 32 * kRowsSteps<END>;
    // (the number of warps is part of the sums' order: the plain linear layer keeps its)
    const int most = END == FpEnd::Linear ? kRowsWarps : kRowsWarps / 2;
    const int warps = std::min(most, std::max(1, (IC + STEP - 1) / STEP));
    const bool vec = IC % 8 == 0 && fp_tma_rows(x, ldx, B, IC) && fp_tma_rows(W, ldw, OC, IC) &&
                     (!W2 || fp_tma_rows(W2, ldw2, OC, IC));
    launch_pdl(vec ? k_fp_rows<END, NT, true> : k_fp_rows<END, NT, false>, (OC + 15) / 16, warps * 32, 0, s,
               static_cast<const uint16_t*>(x), ldx, static_cast<const uint16_t*>(W), ldw,
               static_cast<const uint16_t*>(W2), ldw2, B, IC, OC, e, more);
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
