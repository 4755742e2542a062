// The 16-bit float products of the float layers: what their epilogue does, and how they are run.
#pragma once

#include "ito_float.cuh"

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

// What happens to a product's sums:
//   Linear    FpEpilogue as above
//   Gated     two products of one A: y = act(zg) zu with zg = sum + bias, zu = sum2 + bias2, which go to z and z2
//   Loss      each tile's part of a row's softmax sums, and the row's target among the sums: nothing else is written
//   DLogits   y = (g_loss + g_lse) exp(sum - lse) - g_loss [column is the target], times *scale
//   Grad      y = *alpha sum + acc; the operands may come in two halves (below)
enum class FpEnd { Linear, Gated, Loss, DLogits, Grad };

// the other ends' arguments
struct FpMore {
    const void* bias2;       // Gated
    void* z2;
    int64_t ldz2;
    const int32_t* targets;  // Loss, DLogits: [M], classes; a product's column 0 is class `first` of `classes`
    int first, classes;
    float2* part;            // Loss: [fp_loss_parts()][M] (largest sum, sum of exp(sum - largest))
    float* hit;              // Loss: [M] the target's sum
    const float* lse;        // DLogits: [M]; g_lse and scale may be null
    const float* g_loss;
    const float* g_lse;
    const float* scale;
    const float* alpha;      // Grad: may be null (1)
    const float* acc;        // Grad: [M][ldacc], may be null (0); may be y
    int64_t ldacc;
    void* y2;                // Grad with two halves of rows
    int64_t ldy2;
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
    FpEnd end;
    FpMore x;
    // Gated: the second product's B. Grad: with k_half, B(n, k) = B2(n, k - k_half) from k = k_half on (a
    // multiple of 64; A has 2 k_half columns; each half of B has k_rows rows, and A's columns beyond are 0).
    FpOperand B2;
    int k_half, k_rows;
    // Grad: with a_half, a second result y2 [M][N] from the rows a_half + m of A (an MN-major one; a
    // multiple of 8)
    int a_half;
    // DLogits of a piece of the columns: how many there are in all (0: N). The plan is that of the whole, which
    // the Loss had, so that the sums are the same in every bit.
    int plan_n;
};

// One or two products that do not depend on one another and have the same end (two: Linear or Grad), on the
// tensor cores; ws: the sum of the bytes that fp_gemm_ws_bytes names for each (sums of a product cut into
// slices of K; b_mn: B.mn; halves: 2 for Grad with a_half; plan_n as a product's), 256-byte aligned.
size_t fp_gemm_ws_bytes(int M, int N, int K, bool b_mn, FpEnd end = FpEnd::Linear, int halves = 1,
                        int plan_n = 0);
int fp_gemm(const FpProduct* products, int n, void* ws, cudaStream_t s);
// Parts of each row's sums that a Loss product leaves; 0: none, the workspace's slices are summed and (hit, part[0])
// are the row's own
int fp_loss_parts(int M, int N, int K);

// Gradients of a product of a few rows (fp_few_grad_rows) with one weight or two of [V][D]; g: [B][V], rows on
// 16-byte boundaries and padded to 64 elements, of which those from V on may hold anything.
struct FpFewGrad {
    const uint16_t* g[2];                    // (g[1] null: one weight)
    int64_t ldg;
    const uint16_t* W[2];
    int64_t ldw[2];
    const uint16_t* x;                       // [B][D]
    int64_t ldx;
    int type, out_type, B, V, D;
    const float* alpha;                      // factor of all results; may be null (1)
    void* dx;                                // [B][D] in type: sum over the weights of g W; may be null
    int64_t lddx;
    void* dW[2];                             // [V][D] in out_type: g^T x; both may be null
    int64_t lddw[2];
};
bool fp_few_grad_rows(int B);
size_t fp_few_grad_ws_bytes(int B, int V, int D, int weights);
int fp_few_grad(const FpFewGrad& p, void* ws, cudaStream_t s);

// ---- shared by the layers' entry points (ito_fp_linear.cu)

// Rows whose starts TMA cannot address, copied to rows padded to 32 elements; up to three tensors
// (blockIdx.z).
constexpr int kFpCopies = 3;
struct FpCopy {
    const uint16_t* src[kFpCopies];
    uint16_t* dst[kFpCopies];
    int64_t ld[kFpCopies], ldd[kFpCopies];
    int rows[kFpCopies], cols[kFpCopies];
    Divider by[kFpCopies];                   // by eights of a row
    int n;
};
// Whether the words of all eights of the rows first .. last (Eight16: an element before the eight and one behind
// it at most) lie in the tensor's span of memory.
__host__ __device__ inline bool fp_copy_inner(int64_t first, int64_t last, int rows, int cols, int64_t ld)
{
    return first > 0 && last * ld + (cols + 7) / 8 * 8 < (int64_t)(rows - 1) * ld + cols;
}
int64_t fp_row_stride(int64_t ld, int rows, int cols);           // (a row's stride says nothing about a single row)
bool fp_tma_rows(const void* p, int64_t ld, int rows, int cols);
size_t fp_copy_bytes(const void* p, int64_t ld, int rows, int cols);
// The operand itself, or where its aligned copy will be (at *ws, which moves on), noted in `c`.
const void* fp_aligned_operand(const void* p, int64_t* ld, int rows, int cols, char** ws, FpCopy* c);
int fp_run_copies(const FpCopy& c, cudaStream_t s);
int fp_check_sizes(int B, int IC, int OC);
int fp_check_tensor(const void* p, int type, int64_t ld, int rows, int cols, const char* name);
int fp_check_types(int type, int out_type, int act);
int fp_check_ws(const void* ws, size_t bytes, size_t need);
inline int64_t pad4(int64_t n) { return (n + 3) & ~int64_t(3); }
inline size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// Whether a few rows of x stream W (see ito_fp_rows.cuh) instead of taking tensor-core tiles: the plain linear
// layer's rule, the gated layer's (OC: of one of its two weights; vec: fp_rows_vec of all operands), and that of logits.
bool fp_rows_kernel(int B, int IC, int OC);
bool fp_few_rows(int B, int IC, int OC, bool vec);
bool fp_few_logits(int B, int IC, int OC, bool vec);
// Whether x's and W's rows start on 16-byte boundaries and end with 16 bytes.
bool fp_rows_vec(const void* x, int64_t ldx, const void* W, int64_t ldw, int B, int IC, int OC);

}  // namespace ito
