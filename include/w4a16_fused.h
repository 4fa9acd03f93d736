/*
 * w4a16_fused -- operators around the packed INT4 linear layer (w4a16.h), sm_100a.
 *
 *   w4a16_linear_fused     Y  = act(X . W_hat^T + bias) + residual
 *   w4a16_gated            H  = act(X . Wg_hat^T) * (X . Wu_hat^T)      (gated feed-forward projection)
 *   w4a16_linear_dx        dX = dY . W_hat                              (the layer's input gradient)
 *   w4a16_gated_backward   dX = [dG | dU] . [Wg_hat; Wu_hat],  dG = dH * U * act'(G),  dU = dH * act(G)
 *
 * The packed weights are constants: there is no gradient of codes, scales or
 * zero points (training with frozen weights: adapters, prompts, other layers).
 *
 * Conventions (status codes, alignment, streams, ownership, no allocation,
 * host-side validation, the device fault word) are those of w4a16.h, and so
 * are the weight layouts: qweight uint32 [N][K/8], scales bf16 [N][K/group],
 * zeros int32 [N][K/group], group 32, 64 or 128, K a multiple of 128, any
 * M >= 1 and N >= 1.  Sums and epilogues are computed in FP32 and every
 * output is rounded to BF16 once, from FP32.  Inputs must be finite; every
 * finite BF16 value is accepted.  The same call on the same inputs gives the
 * same bits.
 *
 * Operands.  Up to 16 tokens on the integer GEMVs (see w4a16_linear_fused)
 * weights are exact and activations off by at most 2^-18 of their group's
 * largest.  The GEMM takes both operands in FP16, scaled by a power of two
 * per weight row and per token:
 *   - a weight (q - z) s is off by at most 2^-11 of itself, or 2^-40 |q - z|
 *     of its row's size where that is more.  The size is the largest of its
 *     groups' |s| max(|z|, |15 - z|), each factor raised to a power of two;
 *   - a token's value is exact, or off by 2^-39 of the token's largest value
 *     where that is more; backward, of the token's largest |dY| times the
 *     size of the weight's row.  dG and dU: see w4a16_gated_backward.
 * A group or row of zeros (every code its zero point, or a scale of 0) has no
 * size: backward a row of zeros counts for nothing, and a group of zeros can
 * raise its row's size to at most 2^4 times its smallest group's.
 *
 * Workspaces follow w4a16.h's rule: the first 256 KB hold counters that are
 * zero before first use (w4a16_workspace_init) and left zero by every
 * completed call, so one workspace can serve all calls of the library that
 * are ordered on one stream, captured graphs among them.  Calls that may
 * overlap need a workspace each, and so do, as in w4a16.h, forward calls on
 * up to 16 tokens with N > 8,388,480, whose counters lie beyond that area.
 */
#ifndef W4A16_FUSED_H
#define W4A16_FUSED_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations.  GELU = x Phi(x); GELU_TANH = x / 2 (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))); the derivative of
 * RELU at 0 is 0. */
typedef enum {
    W4A16_ACT_NONE = 0,
    W4A16_ACT_RELU = 1,
    W4A16_ACT_SILU = 2,
    W4A16_ACT_GELU = 3,
    W4A16_ACT_GELU_TANH = 4
} w4a16_act;

/* Bytes of device workspace for w4a16_linear_fused and w4a16_gated on up to M tokens (N: weight rows), 0 for an invalid
 * shape.  Several layers share a workspace of the largest of their sizes. */
W4A16_API size_t w4a16_fused_workspace_bytes(int64_t M, int64_t N, int64_t K, int group);

/* Bytes of device workspace for w4a16_linear_dx and w4a16_gated_backward on up to M tokens (N: weight rows), 0 for an
 * invalid shape. */
W4A16_API size_t w4a16_dx_workspace_bytes(int64_t M, int64_t N, int64_t K, int group);

/*
 * The linear layer with its epilogue: Y[m][n] = act(sum_k X[m][k] W_hat[n][k] + bias[n]) + residual[m][n].
 *   X         device, bf16 bits [M][K]
 *   inv_s     device, fp32 [K], or NULL: AWQ inverse channel scales, X[m][k] is first replaced by
 *             bf16(X[m][k] * inv_s[k]) (as w4a16_linear_awq; any group size)
 *   bias      device, bf16 bits [N], or NULL
 *   act       w4a16_act
 *   residual  device, bf16 bits [M][N], or NULL; may be Y itself (accumulating in place), else must not
 *             overlap Y
 *   Y         device, bf16 bits [M][N]        (written)
 *   workspace device, >= w4a16_fused_workspace_bytes(M, N, K, group) bytes
 * Kernels: one token (K a multiple of 1024, or of 512 for groups of 32 and 64 without inv_s) and 2-16 tokens
 * (groups of 128, K a multiple of 1024) run the integer GEMVs of w4a16_linear with the epilogue in their split-K
 * reduction; everything else runs a tcgen05 GEMM on FP16 operands with the epilogue on its accumulators.
 */
W4A16_API int w4a16_linear_fused(const uint16_t* X, const float* inv_s, int64_t M, int64_t K, int group,
                                 const uint32_t* qweight, const uint16_t* scales, const int32_t* zeros, int64_t N,
                                 const uint16_t* bias, int act, const uint16_t* residual, uint16_t* Y,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * The gated feed-forward projection.  The packed weight holds I = N / 2 gate rows and then I up rows (the gate+up
 * layer): with G[m][j] = sum_k X[m][k] W_hat[j][k] and U[m][j] = sum_k X[m][k] W_hat[I + j][k],
 *   H[m][j] = act(G[m][j]) * U[m][j].
 *   N         weight rows, even
 *   H         device, bf16 bits [M][N / 2]    (written)
 *   GU        device, bf16 bits [M][N], or NULL: [G | U], what w4a16_gated_backward needs (written)
 *   X, inv_s, act, workspace: as w4a16_linear_fused.
 */
W4A16_API int w4a16_gated(const uint16_t* X, const float* inv_s, int64_t M, int64_t K, int group,
                          const uint32_t* qweight, const uint16_t* scales, const int32_t* zeros, int64_t N, int act,
                          uint16_t* H, uint16_t* GU, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The input gradient of the linear layer: dX[m][k] = inv_s[k] * sum_n dY[m][n] W_hat[n][k] (inv_s NULL: 1; the
 * rounding of X * inv_s in the forward pass is passed straight through).
 *   dY        device, bf16 bits [M][N]
 *   dX        device, bf16 bits [M][K]        (written; must not overlap dY)
 *   workspace device, >= w4a16_dx_workspace_bytes(M, N, K, group) bytes
 */
W4A16_API int w4a16_linear_dx(const uint16_t* dY, int64_t M, int64_t N, int group, const uint32_t* qweight,
                              const uint16_t* scales, const int32_t* zeros, int64_t K, const float* inv_s,
                              uint16_t* dX, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The backward pass of w4a16_gated: dG = dH * U * act'(G) and dU = dH * act(G) from GU = [G | U], then
 * dX[m][k] = inv_s[k] * sum_j (dG[m][j] W_hat[j][k] + dU[m][j] W_hat[I + j][k]) from dG and dU before their rounding
 * to BF16: as FP16 operands, off by 2^-11 of their value or 2^-39 of the token's largest |dH| max(2 |U|, |G|) weighted
 * with the rows' sizes.  (A token whose gradients all stay 2^-24 below that -- every gate shut -- takes the BF16 ones.)
 *   dH        device, bf16 bits [M][N / 2]
 *   GU        device, bf16 bits [M][N], as w4a16_gated wrote it
 *   dGU       device, bf16 bits [M][N]: [dG | dU]   (written; may be GU itself, else must not overlap it)
 *   dX        device, bf16 bits [M][K]              (written; must not overlap the inputs)
 *   other arguments as w4a16_linear_dx.
 */
W4A16_API int w4a16_gated_backward(const uint16_t* dH, const uint16_t* GU, int64_t M, int64_t N, int act, int group,
                                   const uint32_t* qweight, const uint16_t* scales, const int32_t* zeros, int64_t K,
                                   const float* inv_s, uint16_t* dGU, uint16_t* dX, void* workspace,
                                   size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_FUSED_H */
