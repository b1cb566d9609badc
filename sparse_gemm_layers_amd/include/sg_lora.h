/*
 * sg_lora.h -- C ABI of the low-rank adapters of libsg.so: every token of a
 * batch with an adapter of its own (or none) beside a shared projection, and the
 * backward pass.
 *
 * The conventions of sg.h hold (row-major matrices, strides in elements, device
 * memory owned by the caller, asynchronous launches on `stream`, arguments
 * checked on the host before any HIP call, every size at least 1).
 */
#ifndef SPARSE_GEMM_LAYERS_AMD_SG_LORA_H
#define SPARSE_GEMM_LAYERS_AMD_SG_LORA_H

#include "sg.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * sg_lora_gemm -- with e = ids[t],
 *   y[t] = base[t] + scale[e] (x[t] . A_e^T) . B_e^T
 * The inner product x . A^T is a fp32 sum and is not rounded: its scaled value
 * enters the second product as a sum of bf16 parts, two for a bf16 y (2^-16 of the
 * value is left out at most), three for a fp32 y (2^-24).  Infinities and NaN of any operand
 * go where the formula takes them.
 * A token whose id is outside [0, L) has no adapter: its y is base, or 0.  A row of x
 * reaches its own row of y alone, and no adapter but its own.
 *   x     : bf16 [T, K], leading dim ldx;  ids: int32 [T], or NULL: adapter 0 for all
 *   a, b  : bf16 [L, r, K] and [L, N, r], contiguous (a smaller rank is padded with zeros)
 *   scale : fp32 [L], or NULL: 1
 *   base  : SG_F32 or SG_BF16 [T, N], leading dim ld_base, or NULL: 0; may be y itself
 *           (same type and leading dim)
 *   y     : SG_F32 or SG_BF16 [T, N], leading dim ldy
 *   workspace : at least sg_lora_gemm_workspace(T, K, N, r, L) bytes (0: none),
 *           256-byte aligned, in use until the work on `stream` is done
 * No output may overlap an input, but for y that is base.
 * Requires K, N and r multiples of 8, r <= 256, K and N under 2^22, L <= 65535, leading
 * dims at least the row, multiples of 8 and under 2^22, T < 2^22; all arrays 16-byte
 * aligned (ids and scale 4).
 */
int64_t sg_lora_gemm_workspace(int64_t T, int64_t K, int64_t N, int r, int64_t L);

sg_status sg_lora_gemm(int64_t T, int64_t K, int64_t N, int r, int64_t L, const uint16_t* x, int64_t ldx,
                       const int32_t* ids, const uint16_t* a, const uint16_t* b, const float* scale, const void* base,
                       sg_dtype base_dt, int64_t ld_base, void* y, sg_dtype y_dt, int64_t ldy, void* workspace,
                       int64_t workspace_bytes, hipStream_t stream);

/*
 * sg_lora_gemm_backward -- gradients of sg_lora_gemm for dy, the gradient of y: with
 * u = x . A_e^T (computed again) and v = scale[e] dy . B_e,
 *   dx[t] = base[t] + v[t] . A_e,  dA_e = sum_t v[t]^T x[t],
 *   dB_e = scale[e] sum_t dy[t]^T u[t]      over the tokens of adapter e
 * (the gradient of sg_lora_gemm's base is dy itself).  Sums are fp32; u and v enter
 * further products as two bf16 parts, three where grad_dt is SG_F32.  An adapter
 * without tokens gets zeros; tokens without an adapter get dx = base, or 0, and enter
 * no sum.  No result depends on an order that changes between calls.
 *   dy   : bf16 [T, N], leading dim ld_dy
 *   base : bf16 [T, K], leading dim ld_base, or NULL: 0; may be dx itself (same
 *          leading dim): what else contributes to the gradient of x
 *   dx   : bf16 [T, K], leading dim ld_dx, or NULL;  da, db: SG_F32 or SG_BF16 of
 *          the shapes of a and b, contiguous, or both NULL
 *   workspace : at least sg_lora_gemm_backward_workspace(T, K, N, r, L) bytes, as above
 * No output may overlap an input, but for dx that is base.
 * Requires what sg_lora_gemm does, and
 * ceil(max(K, N) / 256) * (2 L ceil(r / 64) + ceil(T / 64)) < 2^24 - 4096: the workgroups of one launch.
 */
int64_t sg_lora_gemm_backward_workspace(int64_t T, int64_t K, int64_t N, int r, int64_t L);

sg_status sg_lora_gemm_backward(int64_t T, int64_t K, int64_t N, int r, int64_t L, const uint16_t* dy, int64_t ld_dy,
                                const uint16_t* x, int64_t ldx, const int32_t* ids, const uint16_t* a,
                                const uint16_t* b, const float* scale, const uint16_t* base, int64_t ld_base,
                                uint16_t* dx, int64_t ld_dx, void* da, void* db, sg_dtype grad_dt, void* workspace,
                                int64_t workspace_bytes, hipStream_t stream);

/*
 * How calls of these sizes go, for tests and measurements; nothing is launched.
 *   sg_lora_gemm_plan, plan[4] : launches (1: both products in one); tokens of one adapter that
 *       are taken at a time; ranks of a workgroup of x . A^T; parts of its sum
 *   sg_lora_gemm_backward_plan, plan[6] : tokens taken at a time and ranks of a workgroup of the
 *       first launch; parts of dy . B and of x . A^T; ranks of a workgroup of dA and dB; parts
 *       of their sums over tokens
 * SG_ERR_NULL, or SG_ERR_SHAPE for sizes that the calls refuse.
 */
sg_status sg_lora_gemm_plan(int64_t T, int64_t K, int64_t N, int r, int64_t L, int32_t* plan);

sg_status sg_lora_gemm_backward_plan(int64_t T, int64_t K, int64_t N, int r, int64_t L, int32_t* plan);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_GEMM_LAYERS_AMD_SG_LORA_H */
