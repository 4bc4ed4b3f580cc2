/*
 * gemm_layer.h -- layer operators of the MI355X (gfx950) dense GEMM library
 * (libdense_gemm_tile_amd.so): the matrix product with bias, activation and
 * residual in its epilogue, its gradients, and the same layer with one weight
 * matrix per expert: tokens sorted by expert, their rows sent out and joined
 * again, and the experts' products. Around them: the layer norm before a layer,
 * the gate that chooses the experts, products whose weights are held in 4 bits,
 * and the cross entropy of the output layer.
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

/* Scores of gemm_gate. */
#define GEMM_SCORE_SOFTMAX 0
#define GEMM_SCORE_SIGMOID 1

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

/*
 * gemm_norm: Y = (X - mean) * rstd * gamma + beta for each row, where mean is
 * the row's mean and rstd = 1 / sqrt(mean of (X - mean)^2 + eps).
 *
 * X, Y      M x N of `dtype` (f16, bf16 or GEMM_DTYPE_F32), N >= 1. Y may be X
 *           itself (same pointer and leading dimension).
 * gamma     N values of `dtype`, or NULL for ones. beta: the same, or NULL for
 *           zeros.
 * eps       finite and >= 0.
 *           (Sums are float32: the differences to the mean count as far as their
 *           squares are numbers of it, up to 1.8e19.)
 * mean,     M float32 values each, written when not NULL (kept for the backward
 * rstd      pass).
 */
GEMM_API int gemm_norm(int64_t M, int64_t N, int dtype, const void* X, int64_t ldx,
                  const void* gamma, const void* beta, float eps, void* Y, int64_t ldy,
                  float* mean, float* rstd, void* stream);

/*
 * gemm_norm_grad: the gradients of gemm_norm from dY. With U = (X - mean) * rstd
 * and H = dY * gamma,
 *   dX = rstd * (H - mean of H - U * mean of (H * U)) + R
 *   dgamma = sum over the rows of dY * U,   dbeta = sum over the rows of dY
 * in float32, the rows in an order that does not depend on the run.
 *
 * R         M x N of `dtype` that is added to dX (the gradient that goes past
 *           the norm on a residual stream), or NULL.
 * dX        NULL when only dgamma and dbeta are wanted; may be dY, X or R itself
 *           (same pointer and leading dimension).
 * dgamma,   N values each, or NULL when not wanted.
 * dbeta
 * workspace gemm_norm_grad_workspace(M, N) bytes on the device, 16-byte aligned,
 *           used until the call's work has run (not read or written when dgamma
 *           and dbeta are both NULL).
 */
GEMM_API int gemm_norm_grad(int64_t M, int64_t N, int dtype, const void* dY, int64_t lddy,
                  const void* X, int64_t ldx, const void* gamma, const float* mean,
                  const float* rstd, const void* R, int64_t ldr, void* dX, int64_t lddx,
                  float* dgamma, float* dbeta, void* workspace, int64_t workspace_bytes,
                  void* stream);

/* Bytes of workspace that gemm_norm_grad needs; 0 for sizes it refuses. */
GEMM_API int64_t gemm_norm_grad_workspace(int64_t M, int64_t N);

/*
 * gemm_gate: the `top` experts of each of T tokens, and their weights, from the
 * logits L (T x E of `dtype`: f16, bf16 or GEMM_DTYPE_F32).
 *
 * score     GEMM_SCORE_SOFTMAX: s[t] = softmax(L[t]); GEMM_SCORE_SIGMOID: s =
 *           1 / (1 + exp(-L)).
 * bias      E float32 values, or NULL for none. Experts are compared by their
 *           key, s + bias; the weights do not contain the bias.
 * groups    >= 1, divides E. Experts form `groups` groups of neighbours. A
 *           group's rank is the sum of its group_top (1 or 2) largest keys, and
 *           only the experts of the top_groups best groups are chosen from.
 *           groups == 1: all of them (top_groups is 1; group_top changes nothing).
 * top       experts a token, at most top_groups * (E / groups), and at most 64.
 * renorm    != 0: the weights of a token's choices are divided by their sum (sigmoid
 *           scores that are all 0 in 64 bits stay 0).
 * scale     a factor of every weight.
 *   ids[T * top]      the chosen experts, by falling key; equal ones by rising
 *                     number (of groups too)
 *   weights[T * top]  scale * s[ids], renormalised if wanted
 *
 * Keys are compared as they come out in 64 bits, so that a choice does not hang
 * on a rounding. Without a bias experts, and groups ranked by one of them
 * (group_top 1), are compared by their logits, whose order the scores have, also
 * where scores are equal to 64 bits. An expert whose logit or bias is -infinity is
 * masked: it is not chosen, and adds nothing to its group's rank (a group of masked
 * experts ranks last). Choices that a token has no expert left for are dropped: id
 * -1 and weight 0, which gemm_route, gemm_combine and gemm_gate_grad leave out. A
 * score of NaN ranks below every number and above masked experts, and reaches the
 * weights.
 *
 * E is at most 1024.
 */
GEMM_API int gemm_gate(int64_t T, int64_t E, int64_t top, int dtype, const void* L, int64_t ldl,
                  int score, const float* bias, int64_t groups, int64_t top_groups,
                  int64_t group_top, int renorm, float scale, int32_t* ids, float* weights,
                  void* stream);

/*
 * gemm_gate_grad: dL (T x E of `dtype`), the gradient of L from the gradients
 * dweights of gemm_gate's weights, for the choices in ids. An id outside [0, E)
 * is a dropped choice, whose gradient is not read; a token without choices gets
 * zeros, and one whose renormalised weights gemm_gate leaves at 0. The gradient does
 * not depend on the bias and the groups except through ids. dL may be L itself
 * (same pointer and leading dimension).
 */
GEMM_API int gemm_gate_grad(int64_t T, int64_t E, int64_t top, int dtype, const void* L,
                  int64_t ldl, int score, int renorm, float scale, const int32_t* ids,
                  const float* dweights, void* dL, int64_t lddl, void* stream);

/*
 * gemm_linear_w4: Y = act(A @ W^T + bias) + R with 4-bit weights,
 *   W[n][k] = scales[n][k / group] * (code[n][k] - zeros[n][k / group]).
 *
 * A         M x K of `dtype` (f16 or bf16).
 * B         the codes, 0 to 15, two to a byte: code[n][k] is the lower (k even)
 *           or upper half (k odd) of byte k / 2 of row n. ldb: codes from one
 *           row to the next, even, at least K.
 * scales    N x ceil(K / group) values of `dtype`, leading dimension lds.
 * zeros     the same for the zero points (any values, 7.5 as well as 8), or NULL
 *           for 8 everywhere.
 * group     codes that share a scale: a multiple of 32. A row has at most 1536
 *           groups.
 * bias, act, R, Y, out_dtype: as in gemm_linear. K == 0 leaves act(bias) + R.
 *
 * The codes' products are summed group by group in float32, and each group's sum
 * is scaled in float32: no weight is rounded. (The sums are of code + 16 and of
 * A's values, whose difference has no value where A holds an infinity: its row of
 * Y is NaN.)
 */
GEMM_API int gemm_linear_w4(int64_t M, int64_t N, int64_t K, int dtype, const void* A, int64_t lda,
                  const void* B, int64_t ldb, const void* scales, const void* zeros, int64_t lds,
                  int64_t group, const void* bias, int act, const void* R, int64_t ldr, void* Y,
                  int64_t ldy, int out_dtype, void* stream);

/*
 * gemm_grouped_w4: gemm_linear_w4 with one W (and bias) per group of consecutive
 * rows, as gemm_grouped is to gemm_linear: G groups, offsets, M rows.
 *
 * stride_b  codes from one group's B to the next (even; 0: one for all).
 * stride_s  elements from one group's scales, and zeros, to the next.
 */
GEMM_API int gemm_grouped_w4(int64_t G, int64_t M, int64_t N, int64_t K, int dtype,
                  const int32_t* offsets, const void* A, int64_t lda, const void* B, int64_t ldb,
                  int64_t stride_b, const void* scales, const void* zeros, int64_t lds,
                  int64_t stride_s, int64_t group, const void* bias, int act, const void* R,
                  int64_t ldr, void* Y, int64_t ldy, int out_dtype, void* stream);

/*
 * gemm_loss: cross entropy of an output layer, for T tokens and a vocabulary of
 * V: with the logits L = X @ W^T,
 *   lse[t] = log(sum over v of exp(L[t][v])),   loss[t] = lse[t] - L[t][labels[t]].
 * The logits are not kept. Calls of more than 64 tokens whose operands come in whole
 * 16-byte pieces (addresses, pitches and H) sum them where they are made; others hold
 * pieces of them in float32.
 *
 * X         T x H, W: V x H, of `dtype` (f16 or bf16). H == 0: all logits are 0.
 * labels    T int32. A token whose label is outside [0, V) has the loss 0.
 * loss, lse T float32 values each; lse is written when not NULL (gemm_loss_grad
 *           reads it).
 * V         >= 1.
 * workspace gemm_loss_workspace(T, V, H) bytes on the device, 16-byte aligned,
 *           used until the call's work has run. The size has room for the float32
 *           pieces whatever the call needs: all T x V, or the more of 2^25 values and
 *           4096 for each token.
 */
GEMM_API int gemm_loss(int64_t T, int64_t V, int64_t H, int dtype, const void* X, int64_t ldx,
                  const void* W, int64_t ldw, const int32_t* labels, float* loss, float* lse,
                  void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that gemm_loss needs; 0 for sizes it refuses. */
GEMM_API int64_t gemm_loss_workspace(int64_t T, int64_t V, int64_t H);

/*
 * gemm_loss_grad: the gradients of gemm_loss from dloss (T float32). With
 *   G[t][v] = dloss[t] * (exp(L[t][v] - lse[t]) - (v == labels[t]))
 * (0 for a token whose label is outside [0, V), whose dloss is not read),
 *   dX = G @ W,   dW = G^T @ X.
 * The logits are made again, in pieces of the vocabulary of 2^28 values where they
 * are more, and G is rounded to `dtype`, as the matrix cores read it, before its two
 * products, relative to the largest finite |dloss| of a token that counts: dloss may
 * be of any size (in f16 a token whose |dloss| is below 2^-24 of that loses bits). Of
 * a token whose |dloss| is not that one's, also the label's element is rounded, to
 * half a step of dloss. dX in f16 wants a loss
 * scale all the same, as any gradient in f16.
 *
 * dX        T x H of `dtype`, or NULL when not wanted.
 * dW        V x H of dw_dtype (`dtype` or GEMM_DTYPE_F32), or NULL when not
 *           wanted. accumulate != 0 adds to what dW holds.
 * workspace gemm_loss_grad_workspace(T, V, H) bytes, as above; also for G in 16
 *           bits (all of it, or the more of 2^28 values and 4096 for each token) and
 *           float32 parts of dX.
 */
GEMM_API int gemm_loss_grad(int64_t T, int64_t V, int64_t H, int dtype, const void* X, int64_t ldx,
                  const void* W, int64_t ldw, const int32_t* labels, const float* lse,
                  const float* dloss, void* dX, int64_t lddx, void* dW, int64_t lddw, int dw_dtype,
                  int accumulate, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that gemm_loss_grad needs; 0 for sizes it refuses. */
GEMM_API int64_t gemm_loss_grad_workspace(int64_t T, int64_t V, int64_t H);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_LAYER_H */
