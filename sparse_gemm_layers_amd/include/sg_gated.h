/*
 * sg_gated.h -- C ABI of the gated projections of libsg.so: both projections of
 * a gated feed-forward block, its activation and their product in one kernel,
 * and the backward pass.  bf16 weights as a training program holds them.
 *
 * The conventions of sg.h hold (row-major matrices, strides in elements, device
 * memory owned by the caller, asynchronous launches on `stream`, arguments
 * checked on the host before any HIP call, every size at least 1).
 */
#ifndef SPARSE_GEMM_LAYERS_AMD_SG_GATED_H
#define SPARSE_GEMM_LAYERS_AMD_SG_GATED_H

#include "sg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activation a(g): g / (1 + exp(-g));  g Phi(g), Phi the normal distribution;
 * g sigmoid(2 sqrt(2/pi) (g + 0.044715 g^3));  max(g, 0) with slope 0 at 0. */
typedef int32_t sg_act;
enum { SG_ACT_SILU = 0, SG_ACT_GELU = 1, SG_ACT_GELU_TANH = 2, SG_ACT_RELU = 3 };

/*
 * sg_gated_gemm -- H [T, F] = a(G) * U with
 *   G = X . Wg^T + gate_add,  U = X . Wu^T + up_add
 * G and U are fp32 sums and stay so until H is rounded once.  An addend is what
 * something beside the projection contributes, an adapter's product for one.
 *   x    : bf16 [T, D], leading dim ldx;  gate, up: bf16 [F, D], leading dims ldg, ldu
 *   gate_add, up_add : bf16 [T, F], leading dim ld_add; either may be NULL
 *   h    : SG_F32 or SG_BF16 [T, F], leading dim ldh
 *   g, u : both NULL, or bf16 [T, F], leading dim ld_gu: G and U rounded to bf16, for
 *          the backward pass
 * Requires D and F multiples of 8 and under 2^22, every leading dim at least its
 * row, a multiple of 8 and under 2^22, T < 2^31, ceil(T/128) * ceil(F/64) < 2^22; all
 * arrays 16-byte aligned.
 */
sg_status sg_gated_gemm(int64_t T, int64_t F, int64_t D, const uint16_t* x, int64_t ldx, const uint16_t* gate,
                        int64_t ldg, const uint16_t* up, int64_t ldu, sg_act act, const uint16_t* gate_add,
                        const uint16_t* up_add, int64_t ld_add, void* h, sg_dtype h_dt, int64_t ldh, uint16_t* g,
                        uint16_t* u, int64_t ld_gu, hipStream_t stream);

/*
 * sg_gated_gemm_backward -- gradients of sg_gated_gemm for dh, the gradient of H:
 *   dG = dh * U * a'(G),  dU = dh * a(G)         (and of the addends, which they are too)
 *   dX = dG . Wg + dU . Wu,  dWg = dG^T . X,  dWu = dU^T . X
 * G and U are those kept by the forward pass or, where g and u are NULL, computed
 * again from x, the weights and the addends.  dG and dU are rounded to bf16 once;
 * these values are returned and are the operands of the other three, whose fp32
 * sums are rounded once.  No result depends on an order that changes between calls.
 *   dh, dg, du : bf16 [T, F], leading dims ld_dh, ld_dgu (dg and du)
 *   dx : bf16 [T, D], leading dim ld_dx, or NULL;  dgate, dup: bf16 [F, D], leading dim
 *        ld_dw, or both NULL
 *   workspace : for dx, at least sg_gated_gemm_backward_workspace(T, F, D) bytes (0:
 *        none), 256-byte aligned, in use until the work on `stream` is done
 * Requires what sg_gated_gemm does, and (2 ceil(F/128) + ceil(T/128)) * ceil(D/128) <
 * 2^22.  dg and du may take the place of g and u, no other output that
 * of an input.
 */
int64_t sg_gated_gemm_backward_workspace(int64_t T, int64_t F, int64_t D);

sg_status sg_gated_gemm_backward(int64_t T, int64_t F, int64_t D, const uint16_t* dh, int64_t ld_dh,
                                 const uint16_t* x, int64_t ldx, const uint16_t* gate, int64_t ldg,
                                 const uint16_t* up, int64_t ldu, sg_act act, const uint16_t* g, const uint16_t* u,
                                 int64_t ld_gu, const uint16_t* gate_add, const uint16_t* up_add, int64_t ld_add,
                                 uint16_t* dg, uint16_t* du, int64_t ld_dgu, uint16_t* dx, int64_t ld_dx,
                                 uint16_t* dgate, uint16_t* dup, int64_t ld_dw, void* workspace,
                                 int64_t workspace_bytes, hipStream_t stream);

/*
 * How calls of these sizes go, for tests and measurements; nothing is launched.
 *   sg_gated_gemm_plan : *tokens and *values, the tokens and hidden values of one workgroup of
 *       the forward product, and of that product computed again by the backward call
 *   sg_gated_gemm_backward_plan : *tile, the rows and columns of dx or of a weight's gradient that
 *       one workgroup computes; *parts, those of dx's sum.  More than one take 4 * parts * T * D
 *       bytes of workspace; sg_gated_gemm_backward_workspace is the larger of with and without dw.
 * SG_ERR_NULL, or SG_ERR_SHAPE for sizes that the calls refuse.
 */
sg_status sg_gated_gemm_plan(int64_t T, int64_t F, int64_t D, int32_t* tokens, int32_t* values);

sg_status sg_gated_gemm_backward_plan(int64_t T, int64_t F, int64_t D, int with_dw, int32_t* tile, int32_t* parts);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_GEMM_LAYERS_AMD_SG_GATED_H */
