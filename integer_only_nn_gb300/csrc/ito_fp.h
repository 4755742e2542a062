// The 16-bit float products of the linear layer: what their epilogue does, and how they are run.
#pragma once

#include "ito_internal.h"

namespace ito {

// y = act(sum + bias) + residual; z = sum + bias where asked for
struct FpEpilogue {
    const void* bias;
    int bias_type, act;
    const void* residual;
    int64_t ldr;
    int type, out_type;    // of the operands and z; of y and residual
    void* y;
    int64_t ldy;
    void* z;               // may be null
    int64_t ldz;
};

// A 16-bit operand: [rows][K] with K contiguous (mn false) or [K][rows] (mn true). Its base is
// 16-byte aligned and ld a multiple of 8 elements.
struct FpOperand {
    const void* p;
    int64_t ld;
    bool mn;
};

// C[m][n] = sum_k A(m, k) B(n, k), m < M, n < N, k < K, through the epilogue
struct FpProduct {
    FpOperand A, B;
    int M, N, K;
    FpEpilogue e;
};

// One or two products that do not depend on one another, on the tensor cores; ws: the sum of the
// bytes that fp_gemm_ws_bytes names for each (sums of a product cut into slices of K; b_mn: B.mn),
// 256-byte aligned.
size_t fp_gemm_ws_bytes(int M, int N, int K, bool b_mn);
int fp_gemm(const FpProduct* products, int n, void* ws, cudaStream_t s);

}  // namespace ito
