/*
 * sg_moe.h -- C ABI of the mixture-of-experts operators of libsg.so: routing
 * of tokens to experts with its gradient, linear layers on dense 4-bit weights
 * with group scales, and the routed gated MLP on such weights.
 *
 * The conventions of sg.h hold (row-major matrices, strides in elements, device
 * memory owned by the caller, asynchronous launches on `stream`, arguments
 * checked on the host before any HIP call, every size at least 1).
 */
#ifndef SPARSE_GEMM_LAYERS_AMD_SG_MOE_H
#define SPARSE_GEMM_LAYERS_AMD_SG_MOE_H

#include "sg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Score of an expert: softmax over the token's logits, or each logit's sigmoid. */
typedef int32_t sg_score;
enum { SG_SCORE_SOFTMAX = 0, SG_SCORE_SIGMOID = 1 };

/* Value of a group of experts: its largest key, or the sum of its two largest. */
typedef int32_t sg_group_score;
enum { SG_GROUP_MAX = 0, SG_GROUP_TOP2 = 1 };

/*
 * sg_moe_route -- the k experts of each token and their weights.
 *   s[t, e]  = softmax_e(l[t, :]) or 1 / (1 + exp(-l[t, e]))
 *   key      = l[t, e] without a bias, s[t, e] + bias[e] with one (the bias
 *              steers the choice only, never the weights)
 *   groups   : with n_group > 1 the experts form n_group runs of E / n_group;
 *              a group's value is its largest key (SG_GROUP_MAX) or the sum of
 *              its two largest s + bias (SG_GROUP_TOP2; s alone without a bias;
 *              a group of one usable expert counts that one); the topk_group
 *              groups of largest value stay.
 *   ids      = the k largest keys that stay, largest first; w = s of those,
 *              divided by their sum if renormalize, times scale.
 * Equal keys (and groups) go to the lower index.  Keys are compared as if
 * computed in 64 bits, so the choice does not depend on fp32 rounding.  Weights are
 * rounded once from 64 bits, except that a softmax's sum may be taken in fp32, which
 * depends on the call's sizes and options: those weights are within 32 steps of 2^-24
 * of their value, and may differ by that between calls of few tokens and of many.
 * A logit of -inf or NaN, or a bias of -inf or NaN, takes its expert out
 * (+inf counts as the largest finite value); where fewer than k experts are
 * left the remaining slots hold id -1 and weight 0.
 *   logits : [T, E] SG_F32 or SG_BF16, leading dim ldl;  bias: fp32 [E] or NULL
 *   ids    : int32 [T, k], weights: fp32 [T, k], both contiguous
 * Requires E <= 1024, 1 <= k <= min(E, 64), n_group <= 64 dividing E, 1 <=
 * topk_group <= n_group, k <= topk_group * E / n_group; every array aligned to its
 * element.
 */
sg_status sg_moe_route(const void* logits, sg_dtype l_dt, int64_t T, int64_t E, int64_t ldl, const float* bias, int k,
                       sg_score score, int n_group, int topk_group, sg_group_score group_score, int renormalize,
                       float scale, int32_t* ids, float* weights, hipStream_t stream);

/*
 * sg_moe_route_backward -- gradient of sg_moe_route's weights with respect to
 * its logits, the choice of experts held fixed: with g = grad[t, :],
 *   softmax              : dl_e = scale p_e (g_e [e chosen] - sum_j g_j p_j)
 *   softmax, renormalised: the same over the chosen experts alone
 *   sigmoid              : dl_e = scale g_e s_e (1 - s_e), chosen e only
 *   sigmoid, renormalised: dl_e = scale r_e (1 - s_e) (g_e - sum_j g_j r_j),
 *                          r = s / sum of the chosen s
 * Slots whose id is outside [0, E) count as empty and their grad is not read
 * into any sum; ids of one token are distinct, as sg_moe_route gives them.
 *   grad : fp32 [T, k], ids: int32 [T, k], both contiguous
 *   logits: as above;  dlogits: [T, E] of the logits' dtype, leading dim ldd,
 *   written fully.
 */
sg_status sg_moe_route_backward(const float* grad, const void* logits, sg_dtype l_dt, int64_t T, int64_t E,
                                int64_t ldl, const int32_t* ids, int k, sg_score score, int renormalize, float scale,
                                void* dlogits, int64_t ldd, hipStream_t stream);

/*
 * sg_w4_packed_bytes -- bytes of the packed form of one N x K 4-bit weight with
 * groups of gc columns: ceil(N/16) * ceil(K/128) * (1024 + 64 * 128 / gc), or -1
 * unless gc is 32, 64 or 128, N >= 1, K >= 1, K % gc == 0, N <= 2^31, K <= 2^24.
 *
 * sg_w4_pack -- L weights of int4 codes and their scales into that form (once,
 * when a model is loaded).  One chunk per 16 rows and 128 columns: the codes as
 * the matrix core reads them, then the scales [group][row]; rows past N and
 * columns past K are zero.
 *   wq     : [N, K/2] bytes, two's-complement codes -8 .. 7, element 2j in the low
 *            nibble of byte j (sg_int4_quant_groupwise writes them); leading dim
 *            ldw and distance between weights w_bs in bytes, multiples of 4
 *   s      : fp32, weight e's row n, group c at s[e * s_bs + n * s_sn + c * s_sk]
 *   packed : L * sg_w4_packed_bytes(N, K, gc) bytes, 16-byte aligned, written fully
 */
int64_t sg_w4_packed_bytes(int64_t N, int64_t K, int gc);

sg_status sg_w4_pack(int64_t L, const uint8_t* wq, int64_t ldw, int64_t w_bs, const float* s, int64_t s_sn,
                     int64_t s_sk, int64_t s_bs, int64_t N, int64_t K, int gc, uint8_t* packed, hipStream_t stream);

/*
 * sg_w4a16_gemm_groupwise_packed -- Y [M, N] = X . W^T + bias on a packed weight:
 *   y[m, n] = bias[n] + sum_c s[n, c] sum_{k in group c} x[m, k] code[n, k]
 * in fp32 (the codes are exact in bf16, scales stay fp32), rounded once to y_dt.
 *   x : bf16 [M, K], leading dim ldx;  bias: fp32 [N] or NULL;  y: SG_F32 or SG_BF16
 * Requires ldx >= K, ldx < 2^22, ldy >= N, M < 2^31, N <= 2^27 - 16, ceil(M/128) *
 * ceil(N/256) < 2^23 (a launch's workgroups), ceil(K/128) * 8 chunks under 2^31
 * bytes; x 16-byte aligned, ldx a multiple of 8, y aligned to its element.
 */
sg_status sg_w4a16_gemm_groupwise_packed(int64_t M, int64_t N, int64_t K, const uint16_t* x, int64_t ldx,
                                         const uint8_t* wpacked, int gc, const float* bias, void* y, sg_dtype y_dt,
                                         int64_t ldy, hipStream_t stream);

/*
 * sg_w4a16_moe_mlp -- the routed gated MLP on packed 4-bit experts:
 *   y[t] = sum_j weights[t, j] * Wd_e (silu(Wg_e x_t) * (Wu_e x_t)),  e = ids[t, j]
 * with silu(g) = g / (1 + exp(-g)).  Products and sums are fp32; the inner
 * activations are rounded to bf16 once, as the down product's operand: SG_F32 results
 * carry that rounding (half a step, 2^-8 of an activation at most).  The k
 * contributions are added in an order that the sizes and ids fix: the same call
 * gives the same bits.  A token may name an expert more than once.
 * Slots whose id is outside [0, E) contribute nothing and their weight is not
 * read into the sum; a token without any gets zeros.
 *   x : bf16 [T, D], ld ldx;  ids: int32 [T, k], weights: fp32 [T, k], contiguous
 *   gate, up : E packed F x D weights one after the other; down: E packed D x F
 *   y : [T, D] SG_F32 or SG_BF16, ld ldy
 *   workspace: at least sg_w4a16_moe_mlp_workspace(T, k, E, D, F) bytes, 256-byte
 *              aligned, in use until the work on `stream` is done
 * Requires E <= 1024, D and F multiples of gc and under 2^22, T * k <= 2^30, T *
 * ldx <= 2^30, (ceil(T k/128) + min(T k, E)) * max(ceil(F/128), ceil(D/256)) < 2^23 (-1
 * from the size query, SG_ERR_SHAPE from the call), ldx >= D and a multiple of 8, ldy
 * >= D and a multiple of 4; x, packed weights 16-byte aligned, y aligned to 4 elements.
 */
int64_t sg_w4a16_moe_mlp_workspace(int64_t T, int k, int64_t E, int64_t D, int64_t F);

sg_status sg_w4a16_moe_mlp(int64_t T, int k, int64_t E, int64_t D, int64_t F, const uint16_t* x, int64_t ldx,
                           const int32_t* ids, const float* weights, const uint8_t* gate, const uint8_t* up,
                           const uint8_t* down, int gc, void* y, sg_dtype y_dt, int64_t ldy, void* workspace,
                           int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_GEMM_LAYERS_AMD_SG_MOE_H */
