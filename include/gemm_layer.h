/*
 * gemm_layer.h -- layer operators of the MI355X (gfx950) dense GEMM library
 * (libdense_gemm_tile_amd.so): the matrix product with bias, activation and
 * residual in its epilogue, its gradients, and the same layer with one weight
 * matrix per expert: tokens sorted by expert, their rows sent out and joined
 * again, and the experts' products.
 *
 * Conventions are those of dense_gemm_tile.h: row-major matrices, leading
 * dimensions in elements, device pointers owned by the caller, work enqueued
 * on `stream` (a hipStream_t; NULL is the default stream), nothing allocated
 * or synchronised, kernel launches only (so calls can be captured into a HIP
 * graph), the GEMM_* return codes, and gemm_last_error() / gemm_last_path()
 * for the calling thread. Sums are held in float32; a 16-bit result is rounded
 * once, to nearest with ties to even.
 *
 * What a call writes must not overlap what it reads, except where an entry
 * below allows it: other overlaps of operands are rejected with
 * GEMM_ERR_ALIAS.
 *
 * Numbers read on the GPU (expert ids, offsets, slots) cannot be checked
 * before the call returns. The kernels check them where they use them: an id
 * outside [0, E) counts as dropped, a slot outside [0, T*top) is skipped, and
 * offsets are clamped to [0, M], so no access leaves the buffers, also where
 * offsets decrease (what such a call computes is not defined).
 *
 * A product of more output tiles than one launch holds (2^32 threads: from 2^22
 * tiles on, by the kernel) is refused with GEMM_ERR_UNSUPPORTED.
 */
#ifndef GEMM_LAYER_H
#define GEMM_LAYER_H

#include <stdint.h>

#include "dense_gemm_tile.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of float32 results and rows, beside GEMM_DTYPE_F16 / _BF16. */
#define GEMM_DTYPE_F32 6

/* Activations. GELU is the tanh form, GELU_ERF the form with the normal
 * distribution function; SILU is z / (1 + exp(-z)). */
#define GEMM_ACT_NONE 0
#define GEMM_ACT_RELU 1
#define GEMM_ACT_GELU 2
#define GEMM_ACT_GELU_ERF 3
#define GEMM_ACT_SILU 4

/*
 * gemm_linear: Z = op(A) @ op(B) + bias,  Y = act(Z) + R.
 *
 * M, N, K   >= 0, transA / transB, lda, ldb, A, B: as in gemm(), with
 *           dtype GEMM_DTYPE_F16 or GEMM_DTYPE_BF16. K == 0 leaves
 *           Z = bias (A and B are not read).
 * bias      N values of `dtype`, or NULL for none.
 * act       one of GEMM_ACT_*.
 * R         M x N of `out_dtype`, or NULL for none. R may be Y itself (same
 *           pointer and ldr == ldy).
 * Y         M x N of `out_dtype`: `dtype` itself or GEMM_DTYPE_F32.
 * Z         M x N of `dtype`, written when not NULL (kept for the backward
 *           pass); the activation is applied to the unrounded sum.
 */
GEMM_API int gemm_linear(int64_t M, int64_t N, int64_t K, int dtype, int transA, int transB,
                const void* A, int64_t lda, const void* B, int64_t ldb, const void* bias, int act,
                const void* R, int64_t ldr, void* Y, int64_t ldy, int out_dtype, void* Z,
                int64_t ldz, void* stream);

/* The host-side checks and kernel choice of gemm_linear() without a launch. */
GEMM_API int gemm_linear_validate(int64_t M, int64_t N, int64_t K, int dtype, int transA, int transB,
                const void* A, int64_t lda, const void* B, int64_t ldb, const void* bias, int act,
                const void* R, int64_t ldr, const void* Y, int64_t ldy, int out_dtype,
                const void* Z, int64_t ldz);

/*
 * gemm_grouped: gemm_linear with one B (and bias) per group of consecutive
 * rows. Rows offsets[g] .. offsets[g+1]-1 of A (stored [M][K]), R, Y and Z
 * belong to group g; rows from offsets[G] on are neither read nor written.
 *
 * G         >= 0 groups; offsets: G + 1 int32 on the device, not decreasing,
 *           offsets[0] == 0 (an empty group has two equal ones).
 * M         rows of A and Y: at least offsets[G].
 * B         group g's matrix starts at B + g * stride_b elements (0: one for
 *           all); transB: it is stored [N][K], else [K][N].
 * bias      group g's N values start at bias + g * N, or NULL.
 */
GEMM_API int gemm_grouped(int64_t G, int64_t M, int64_t N, int64_t K, int dtype, int transB,
                 const int32_t* offsets, const void* A, int64_t lda, const void* B, int64_t ldb,
                 int64_t stride_b, const void* bias, int act, const void* R, int64_t ldr, void* Y,
                 int64_t ldy, int out_dtype, void* Z, int64_t ldz, void* stream);

GEMM_API int gemm_grouped_validate(int64_t G, int64_t M, int64_t N, int64_t K, int dtype, int transB,
                 const int32_t* offsets, const void* A, int64_t lda, const void* B, int64_t ldb,
                 int64_t stride_b, const void* bias, int act, const void* R, int64_t ldr,
                 const void* Y, int64_t ldy, int out_dtype, const void* Z, int64_t ldz);

/*
 * gemm_grouped_grad_weight: D_g = A_g^T @ B_g for each group g, where A_g and
 * B_g are rows offsets[g] .. offsets[g+1]-1 of A (M x N) and B (M x K): the
 * gradient of the group's [N][K] weights with A = dY, B = X, or of its [K][N]
 * weights with A = X, B = dY. A group without rows gives zeros.
 *
 * D         group g's N x K result of out_dtype (`dtype` or GEMM_DTYPE_F32)
 *           starts at D + g * stride_d. accumulate != 0 adds to what D holds.
 */
GEMM_API int gemm_grouped_grad_weight(int64_t G, int64_t M, int64_t N, int64_t K, int dtype,
                 const int32_t* offsets, const void* A, int64_t lda, const void* B, int64_t ldb,
                 void* D, int64_t ldd, int64_t stride_d, int out_dtype, int accumulate,
                 void* stream);

GEMM_API int gemm_grouped_grad_weight_validate(int64_t G, int64_t M, int64_t N, int64_t K, int dtype,
                 const int32_t* offsets, const void* A, int64_t lda, const void* B, int64_t ldb,
                 const void* D, int64_t ldd, int64_t stride_d, int out_dtype, int accumulate);

/*
 * gemm_act_grad: dZ = dY * act'(Z) (all M x N of `dtype`: the operand of the
 * products that follow, dX = dZ W and dW = dZ^T X, which therefore see it rounded
 * once), and per group the bias gradient db[g][n] = sum over the group's rows of
 * the unrounded dZ, in float32, the rows in an order that does not depend on the
 * run.
 *
 * offsets   as in gemm_grouped, or NULL for one group of all M rows (G == 1).
 * Z         not read when act is GEMM_ACT_NONE (may be NULL).
 * dZ        NULL when only db is wanted; may be dY or Z itself (same pointer
 *           and leading dimension). db: G x N, or NULL when only dZ is wanted.
 * workspace device memory of at least gemm_act_grad_workspace(G, M, N) bytes,
 *           16-byte aligned, used until the call's work has run (not read or
 *           written when db is NULL).
 */
GEMM_API int gemm_act_grad(int64_t G, int64_t M, int64_t N, int dtype, int act, const int32_t* offsets,
                  const void* dY, int64_t lddy, const void* Z, int64_t ldz, void* dZ, int64_t lddz,
                  float* db, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that gemm_act_grad needs; 0 for sizes it refuses. */
GEMM_API int64_t gemm_act_grad_workspace(int64_t G, int64_t M, int64_t N);

/*
 * gemm_route: sorts the T * top choices of T tokens by expert, keeping the
 * order of choices within an expert. ids: T x top int32 (any value outside
 * [0, E) means dropped).
 *   offsets[E + 1]   first sorted position of each expert; offsets[E] is the
 *                    number of choices kept
 *   order[T * top]   the choice (t * top + j) at each sorted position; the
 *                    dropped ones follow the kept ones, in their own order
 *   slot[T * top]    the sorted position of each choice, -1 for a dropped one
 * E is at most 1024. workspace: gemm_route_workspace(T, top, E) bytes on the
 * device, 16-byte aligned (NULL when that is 0).
 */
GEMM_API int gemm_route(int64_t T, int64_t top, int64_t E, const int32_t* ids, int32_t* offsets,
               int32_t* order, int32_t* slot, void* workspace, int64_t workspace_bytes,
               void* stream);

GEMM_API int64_t gemm_route_workspace(int64_t T, int64_t top, int64_t E);

/*
 * gemm_dispatch: Xs[slot[t][j]] = X[t] for every kept choice. X: T x H,
 * Xs: (T * top) x H, both of `dtype` (f16, bf16 or GEMM_DTYPE_F32); rows of Xs
 * that no slot names are not written. Rows of more than 65535 * 256 accesses (of 16
 * bytes, or as few as H, the addresses and the pitches allow) are refused.
 */
GEMM_API int gemm_dispatch(int64_t T, int64_t top, int64_t H, int dtype, const void* X, int64_t ldx,
                  const int32_t* slot, void* Xs, int64_t ldxs, void* stream);

/*
 * gemm_combine: Y[t] = sum over j of weights[t][j] * Ys[slot[t][j]], plus
 * R[t], choices in order, dropped ones left out. weights: T x top float32, or
 * NULL for ones (which makes this the gradient of gemm_dispatch). R: T x H or
 * NULL; it may be Y itself.
 */
GEMM_API int gemm_combine(int64_t T, int64_t top, int64_t H, int dtype, const void* Ys, int64_t ldys,
                 const int32_t* slot, const float* weights, const void* R, int64_t ldr, void* Y,
                 int64_t ldy, void* stream);

/*
 * gemm_combine_grad: dYs[slot[t][j]] = weights[t][j] * dY[t] and
 * dweights[t][j] = <dY[t], Ys[slot[t][j]]> (0 for a dropped choice). Either
 * output may be NULL; Ys is not read without dweights. dYs may be Ys itself.
 * The gradient of R is dY.
 */
GEMM_API int gemm_combine_grad(int64_t T, int64_t top, int64_t H, int dtype, const void* dY, int64_t lddy,
                      const void* Ys, int64_t ldys, const int32_t* slot, const float* weights,
                      void* dYs, int64_t lddys, float* dweights, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_LAYER_H */
