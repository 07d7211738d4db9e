/*
 * fp8bs_layer.h -- what stands around the FP8 products of a mixture-of-experts
 * block: the residual's addition and RMS norm with an FP8 output, the router's
 * choice of experts, their gradients, and the experts themselves for few
 * tokens.  Part of the library that fp8bs.h declares; its formats, quantization
 * rule and conventions (device pointers, streams, argument checks and their
 * order, status codes, nothing allocated or kept) hold here too.  Scalars are
 * checked with the flags (FP8BS_ERR_FLAGS); two queries of workspace sizes and one of
 * tiles run on the host alone.
 */
#ifndef FP8BS_LAYER_H
#define FP8BS_LAYER_H

#include "fp8bs.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of norm weights and router logits. */
enum { FP8BS_BF16 = 0, FP8BS_FP32 = 1 };

/* Flag of the routing calls: the weights of a token's chosen experts sum to 1
 * (a softmax over the chosen logits).  Without it they are the softmax over all
 * of the token's logits. */
enum { FP8BS_ROUTE_RENORM = 4u };

/*
 * Residual addition, RMS norm and 1x128 quantization:
 *   h    = RN_bf16(x + residual)            (h = x where residual is NULL)
 *   rstd = 1 / sqrt(mean over k of h[m][k]^2 + eps)
 *   y    = h weight[k] rstd                 in FP32
 *   q, s = the 1x128 quantization of y (the rule of fp8bs.h), as the A operand
 *          of the GEMMs takes it
 *   x, residual : BF16 [M][K]
 *   weight      : [K], weight_type FP8BS_BF16 or FP8BS_FP32
 *   h           : BF16 [M][K]; NULL where residual is NULL.  May be x or
 *                 residual (in place); otherwise no output overlaps an input.
 *   y           : BF16 [M][K] (y rounded once), or NULL
 *   q, s        : E4M3 [M][K], FP32 [K/128][M]
 *   rstd        : FP32 [M], or NULL
 *   flags       : 0 or FP8BS_SCALE_POW2
 * The sum of squares and y are FP32: they have to stay below 2^128 in size, and
 * h weight below 2^144.  Inputs must be finite.
 * Requires 0 <= M < 2^31, 0 < K <= 16384, K % 128 == 0, eps >= 2^-126 and
 * finite; residual and h both given or both NULL (else FP8BS_ERR_NULL).
 */
fp8bs_status fp8bs_rms_norm_quantize(const void* x, const void* residual, const void* weight, int32_t weight_type,
                                     float eps, int64_t M, int64_t K, void* h, void* y, uint8_t* q, float* s,
                                     float* rstd, uint32_t flags, fp8bs_stream_t stream);

/*
 * Gradients of that norm, the quantization passed through unchanged:
 *   n  = h rstd,  g = dy weight[k]
 *   dx = RN_bf16(dh + rstd (g - n mean over k of (g n)))   (both x and residual)
 *   dweight[k] (+)= sum over m of dy n
 *   dy, h  : BF16 [M][K];  rstd : FP32 [M];  weight as above
 *   dh     : BF16 [M][K], what reaches h by other ways, or NULL (none)
 *   dx     : BF16 [M][K]; may be dy or dh (in place)
 *   dweight: FP32 [K]; accumulate = 1 adds to its contents, 0 overwrites them
 *            (with 0 where M is 0)
 *   workspace : fp8bs_rms_norm_backward_workspace bytes (NULL if 0), contents
 *               overwritten; calls that share it must not overlap in time
 * n, g and the sums are FP32: they have to stay below 2^128 in size, and keep fewer
 * bits below 2^-126.  The order is fixed: the same inputs give the same bits.
 * Requires M and K as above, accumulate in {0, 1} (else FP8BS_ERR_FLAGS).
 */
fp8bs_status fp8bs_rms_norm_backward(const void* dy, const void* h, const float* rstd, const void* weight,
                                     int32_t weight_type, const void* dh, int64_t M, int64_t K, void* dx,
                                     float* dweight, int32_t accumulate, void* workspace, int64_t workspace_bytes,
                                     fp8bs_stream_t stream);

/* Workspace bytes of fp8bs_rms_norm_backward (bytes: HOST pointer). */
fp8bs_status fp8bs_rms_norm_backward_workspace(int64_t M, int64_t K, int64_t* bytes);

/*
 * The router's choice: for each token the topk experts with the largest logits,
 * in falling order (ties: the lowest index), and their weights
 *   exp(logit) / sum of exp(logit)   over the chosen experts with
 *                                    FP8BS_ROUTE_RENORM, else over all E
 * An expert whose logit is -inf or NaN is left out: it adds nothing and is never
 * chosen.  Where fewer than topk experts are left the remaining places get id -1
 * and weight 0.  Logits of +inf share the weight evenly among themselves.
 *   logits  : [T][E], logits_type FP8BS_BF16 or FP8BS_FP32
 *   ids     : INT32 [T][topk],  weights : FP32 [T][topk]
 * Requires 0 <= T < 2^31, 0 < E <= 1024, 0 < topk <= min(E, 64).
 */
fp8bs_status fp8bs_moe_route(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t topk,
                             int32_t* ids, float* weights, uint32_t flags, fp8bs_stream_t stream);

/*
 * Gradient of the weights with respect to the logits, the choice held fixed:
 *   p_i = the softmax over the chosen logits (FP8BS_ROUTE_RENORM) or over all
 *   dlogits[t][i] = p_i (G_i - sum over j of p_j G_j), G_i the sum of dweights
 *                   over the places with id i; with FP8BS_ROUTE_RENORM a place
 *                   counts as often as it stands in ids
 *   logits  : as given to fp8bs_moe_route;  ids : INT32 [T][topk], its output
 *   dweights: FP32 [T][topk];  dlogits : [T][E], the logits' type
 * Ids outside [0, E) and experts whose logit is -inf or NaN have no part.
 * Sizes as above.
 */
fp8bs_status fp8bs_moe_route_backward(const void* logits, int32_t logits_type, const int32_t* ids,
                                      const float* dweights, int64_t T, int32_t E, int32_t topk, void* dlogits,
                                      uint32_t flags, fp8bs_stream_t stream);

/*
 * The experts of a few tokens (decoding):
 *   g, u   = the first and last I rows of w13[e] times x[t]
 *   out[t] = sum over j of w2[e] (weights[t][j] g / (1 + exp(-g)) u), e = ids[t][j]
 *   x      : E4M3 [T][H],      sx  : FP32 [H/128][T]              (1x128 tiles)
 *   ids    : INT32 [T][topk];  weights : FP32 [T][topk].  Places with an id
 *            outside [0, E) are left out; an expert that stands twice in a row
 *            counts once with the sum of its weights.
 *   w13    : E4M3 [E][2 I][H], s13 : FP32 [E][2 I / 128][H/128]   (128x128 blocks)
 *   w2     : E4M3 [E][H][I],   s2  : FP32 [E][H/128][I/128]
 *   out    : BF16 or FP32 [T][H]; tokens without an expert get 0
 *   workspace : fp8bs_moe_experts_workspace bytes, contents overwritten; calls
 *               that share it must not overlap in time
 * The first product promotes FP8 chunk products as the GEMMs do.  The weighted
 * activations are held as two BF16 parts (2^-17 of a value is lost) and meet the
 * codes of w2, which BF16 holds exactly (parts below 2^-126 may count as 0); sums
 * are FP32, in a fixed order.  A chunk's products are added before their scale: the
 * weighted activations have to stay below 2^112 (2^112 * 448 * 128 < 2^128).
 * Requires 0 <= T <= 128 (more tokens: the grouped GEMMs), 0 < topk <= 16,
 * 0 < E <= 1024, H and I multiples of 128 from 128 to 32768 with 2 H I < 2^31.
 */
fp8bs_status fp8bs_moe_experts(const uint8_t* x, const float* sx, const int32_t* ids, const float* weights,
                               const uint8_t* w13, const float* s13, const uint8_t* w2, const float* s2, void* out,
                               int64_t T, int64_t H, int64_t I, int32_t E, int32_t topk, int32_t out_dtype,
                               void* workspace, int64_t workspace_bytes, fp8bs_stream_t stream);

/* Kernels that a fp8bs_moe_experts call of these sizes would run on (host-side
 * query for tests and tuning): rows that one pass over an expert's weights serves
 * (16 or 64), columns of a workgroup in the first and in the second product, and
 * the waves that share them in the second (8: those of all experts at once, so
 * that no sum over experts is left).  HOST pointers. */
fp8bs_status fp8bs_moe_experts_tile(int64_t T, int64_t H, int64_t I, int32_t E, int32_t topk, int32_t* rows,
                                    int32_t* up_columns, int32_t* down_columns, int32_t* down_waves);

/* Workspace bytes of fp8bs_moe_experts (bytes: HOST pointer). */
fp8bs_status fp8bs_moe_experts_workspace(int64_t T, int64_t H, int64_t I, int32_t E, int32_t topk, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* FP8BS_LAYER_H */
