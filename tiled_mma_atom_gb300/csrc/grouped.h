// grouped.h — arguments of the expert-grouped products and of the dense
// product with the residual epilogue, as their kernels take them.
#pragma once

#include "internal.h"

namespace tmg {

// What follows the sum z = (A . B^T) in the epilogue, in fp32:
//   z *= scale_a[row of A] * scale_b[n], z += bias[n]; preact = bf16(z);
//   D = bf16(act(z) + residual).
// swiglu: z has 2 F columns, D = silu(z[f]) z[F + f]; preact holds both halves.
// swiglu_grad: z is the gradient of a SwiGLU result, preact (an input) holds
// its two halves; D (2 F columns) their gradients.
struct ProductEpi {
    const float *scale_a;
    const float *scale_b;      // (E, rows of B)
    const float *bias;         // dense product only
    const void *residual;      // bf16, dense product only
    void *preact;              // bf16: written, or read by swiglu_grad
    int64_t ld_residual, ld_preact;
    int act;                   // kAct*
};

// D[r] = A[rows ? rows[r] : r] . B[e]^T for offsets[e] <= r < offsets[e + 1]
// (offsets null: one group of all R rows).
struct GroupedArgs {
    const void *A, *B;
    void *D;
    int64_t R;                 // rows of D (and of A without `rows`)
    int64_t T;                 // rows of A
    int64_t N, K, E;           // rows of each expert's B, contraction, experts
    int64_t lda, a_col, ldd;   // strides in elements; D has unit column stride
    int64_t b_expert, b_row, b_col;
    const int32_t *offsets, *rows;
    bool e4m3;
    ProductEpi epi;
};

// Copy of an operand with 16-byte rows: dst[e][r][k], r < rows_p, k < Kp, of
// src[e s_e + r s_row + k s_col]; zeros for r >= rows and k >= K.
struct Pack3Args {
    const void *src;
    void *dst;
    int64_t E, rows, K, s_e, s_row, s_col;
    int64_t rows_p, Kp, d_e;
};
cudaError_t launch_pack3(const Pack3Args &a, int elem, int num_sms, cudaStream_t s);
// dst[r] = src[numbers[r]] (zeros where that is not one of src_rows): rows of
// `bytes` bytes, all addresses and strides multiples of 16, dst zero-padded to
// dst_stride.
cudaError_t launch_gather_rows(const void *src, int64_t stride, int64_t src_rows, int64_t bytes, const int32_t *numbers,
                               int64_t rows, void *dst, int64_t dst_stride, int num_sms, cudaStream_t s);

// dB[e][n][k] = sum over the rows r of group e of dD[r][n] A[rows ? rows[r] : r][k].
struct WgradArgs {
    const void *dD, *A;
    void *dB;                  // (E, N, K) contiguous
    int64_t R, T, N, K, E;
    int64_t ldd, d_col, lda, a_col;
    const int32_t *offsets, *rows;     // offsets null: one group of all R rows
};
// ------------------------------------------------------------- routing
struct RouteArgs {
    const void *logits;
    bool bf16;
    int64_t T, ld;
    int E, k;
    bool normalize;
    float *weights;
    int32_t *experts, *offsets, *rows, *slots;
    uint16_t *counts;          // workspace: route_counts_bytes()
};
size_t route_counts_bytes(int64_t T, int E, int num_sms);
cudaError_t launch_route(const RouteArgs &a, int num_sms, cudaStream_t s);
cudaError_t launch_route_backward(const void *logits, bool bf16, int64_t T, int64_t ld, int E, int k, bool normalize,
                                  const int32_t *experts, const float *dweights, void *dlogits, int num_sms,
                                  cudaStream_t s);
struct CombineArgs {
    const void *Y;             // bf16 (R, H), row stride ldy
    const int32_t *slots;      // (T, k)
    const float *weights;      // (T, k) or null (ones)
    const void *residual;      // bf16 (T, H) or null
    void *out;                 // bf16 (T, H)
    int64_t T, H, R, ldy, ldr, ldo;
    int k;
};
cudaError_t launch_combine(const CombineArgs &a, cudaStream_t s);
struct CombineGradArgs {
    const void *dOut, *Y;      // bf16 (T, H), (R, H)
    const int32_t *slots;
    const float *weights;      // or null (ones)
    void *dY;                  // bf16 (R, H) contiguous
    float *dweights;           // (T, k) or null
    int64_t T, H, R, ldo, ldy;
    int k;
};
cudaError_t launch_combine_backward(const CombineGradArgs &a, cudaStream_t s);

// --------------------------------------- gradient of the dense product
// dz = bf16(dD act'(preact)) (M, N) contiguous; column sums of the fp32 dz in
// dbias through `partials` (act_grad_chunks(M, N) x N fp32).  act none: only the
// sums (dz null).  dbias null: only dz.
int act_grad_chunks(int64_t M, int64_t N);
cudaError_t launch_act_grad(const void *dD, int64_t ldd, const void *preact, int64_t ldp, int act, int64_t M, int64_t N,
                            void *dz, float *partials, float *dbias, cudaStream_t s);

}  // namespace tmg
