/*
 * moe355_block.h -- C ABI of the operators that stand around the MoE layer of moe355.h in a
 * transformer block, in the same library (libmoe355.so): the residual's addition with the
 * RMS norm and its 8-bit output, the router's choice of experts, the dispatch of rows that
 * are 8-bit codes already, and the expert FFN of a few tokens with MXFP4 weights.
 *
 *   serving, one token:  moe_rmsnorm -> (router logits) -> moe_router_topk -> moe_expert_ffn_decode
 *   serving, a prompt:   moe_rmsnorm -> (router logits) -> moe_router_topk -> moe_plan ->
 *                        moe_dispatch_quantized -> moe_expert_ffn -> moe_combine
 *   training:            the bf16 forms of these; moe_combine_backward's d_topk_weights go to
 *                        moe_router_topk_backward, the block's dx to moe_rmsnorm_backward
 *
 * The conventions are those of moe355.h (caller-owned device memory of the current device,
 * asynchronous on `stream`, argument errors before anything is enqueued, no allocation, no
 * synchronisation, dense row-major arrays, bf16 and OCP E4M3). Besides:
 *   - Arrays of bf16 and of 8-bit codes, the packed weights, the norm's weight and the
 *     workspaces are 16-byte aligned, arrays of 4-byte values 4-byte aligned; anything else
 *     is MOE_ERR_INVALID.
 *   - T = 0 is a call with nothing to do: MOE_OK, with the row arrays not looked at (they may
 *     be null). T < 0 is MOE_ERR_INVALID.
 *   - Arrays written may not overlap arrays read, except where a call says so.
 *   - Workspaces hold nothing between calls and need no initialisation. Calls that may run at
 *     the same time (two streams, two captured graphs) need one each.
 *
 * Quantised rows ("q", "q_s") are the layer's activation formats with row-major scales:
 * e4m3 codes [T][H], and ceil(H/128) 4-byte scale words a row: MOE_FP8_E4M3_G128 one fp32
 * scale per 1x128 group (H % 128 == 0), MOE_MXFP4 (MXFP8 activations) the four E8M0 bytes
 * of the group's 1x32 blocks, in order (H % 32 == 0; bytes past the row's last block are 0).
 * A group or block that holds a NaN or an infinity has the scale NaN (E8M0 255) and zero
 * codes, so that all of its values are NaN.
 */
#ifndef MOE355_BLOCK_H
#define MOE355_BLOCK_H

#include "moe355.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of the norm's weight and of the router's logits: MOE_BF16 or this. */
enum { MOE_F32 = 16 };

/*
 * Root-mean-square norm of every row, with the residual's addition in front:
 *   s[t]    = bf16(x[t] + res[t])   (res null: s = x)
 *   rstd[t] = fp32(1 / sqrt(mean(s[t]^2) + eps))          sums and root in 64 bits
 *   y[t]    = bf16((s[t] * rstd[t]) * weight)             fp32 products, rounded one by one
 *   q, q_s  = the quantised row y[t] in format q_dtype: the same codes and scales, bit for
 *             bit, that moe_dispatch makes of y (finite rows)
 * x, res, s_out, y: bf16 [T][H]; weight: bf16 or fp32 [H] (weight_dtype); rstd: fp32 [T].
 * s_out receives s (needs res; s is what moe_rmsnorm_backward takes); s_out, y, rstd and
 * q with q_s may each be null, but one of y and q is there. q_dtype: MOE_BF16 with q and q_s
 * null, or MOE_FP8_E4M3_G128 or MOE_MXFP4 with both. s_out and y may be x or res (not both
 * the same one): a row is read before it is written. Rows with an infinity have rstd 0.
 * Errors: MOE_ERR_INVALID (null or misaligned pointers, T < 0, H < 8, eps negative or not
 * finite, unknown types, s_out without res, s_out the same array as y), MOE_ERR_UNSUPPORTED
 * (H % 8 != 0 or H > 32768; fp8 with H % 128 != 0; MXFP8 with H % 32 != 0).
 */
MOE355_API int moe_rmsnorm(const void* x, const void* res, const void* weight, int32_t weight_dtype, int32_t T,
                           int32_t H, double eps, void* s_out, void* y, float* rstd, int32_t q_dtype, void* q,
                           void* q_s, void* stream);

/* Bytes of moe_rmsnorm_backward's workspace (0 for invalid sizes or T = 0). */
MOE355_API size_t moe_rmsnorm_backward_workspace_bytes(int32_t T, int32_t H);

/*
 * Backward of moe_rmsnorm's bf16 output, with the gradient of the stream behind the block:
 *   g = dy[t] * weight, xhat = s[t] * rstd[t], c = mean(g * xhat)
 *   dx[t]   = bf16(rstd[t] * (g - xhat * c) + d_res[t])   (d_res null: without it)
 *   dweight = sum over t of dy[t] * xhat                  fp32, in an order that T and H fix
 * dx is the gradient of x and, the same, of res. dy, s, d_res, dx: bf16 [T][H]; s is x, or
 * s_out where there was a residual; dweight: fp32 [H], written (not added to), or null; with
 * T = 0 it is zero-filled. dx may be dy or d_res. ws: the workspace, used for dweight (null
 * if dweight is). Results do not change from run to run.
 * Errors: MOE_ERR_INVALID (null or misaligned pointers, sizes, unknown type, small
 * workspace), MOE_ERR_UNSUPPORTED (H % 8 != 0 or H > 32768).
 */
MOE355_API int moe_rmsnorm_backward(const void* dy, const void* s, const void* weight, int32_t weight_dtype,
                                    const float* rstd, const void* d_res, int32_t T, int32_t H, void* dx,
                                    float* dweight, void* ws, size_t ws_bytes, void* stream);

/* How the router scores experts. */
enum {
  MOE_SCORE_SOFTMAX = 0, /* softmax over a token's experts */
  MOE_SCORE_SIGMOID = 1  /* each expert by itself */
};

typedef struct moe_router_config {
  int32_t score;       /* MOE_SCORE_* */
  int32_t normalize;   /* 1: a token's weights are divided by their sum (softmax: softmax over
                          the chosen experts' logits), 0: they are the scores */
  int32_t groups;      /* the E experts are this many groups of E / groups neighbours (1: none) */
  int32_t topk_groups; /* groups a token may choose from */
  int32_t group_top;   /* a group counts as the sum of its group_top (1 or 2) largest keys */
  float scale;         /* factor of the weights */
} moe_router_config;

/*
 * The K experts of every token and their weights, from the router's logits:
 *   key  = logit; with a bias, or with groups > 1 and group_top = 2, key = score + bias (the
 *          score in 64 bits: softmax over the token's experts, or sigmoid)
 *   the topk_groups groups whose group_top largest keys sum to the most stay (a group with
 *   fewer keys counts those it has); of their experts the K with the largest keys are chosen,
 *   largest first. Ties go to the lower index.
 *   topk_weights = scale * score / (normalize ? sum over the chosen of their scores : 1)
 * bias: fp32 [E] or null; it takes part in the choice alone, not in the weights.
 * Masks: an expert whose logit is -infinity or NaN, or whose bias is, is switched off for the
 * token: never chosen, and (logit) no part of the softmax. The type's lowest value is an
 * ordinary logit. +infinity counts as the largest finite value. A token with fewer than K
 * experts to choose from has topk_idx -1 and weight 0 in the places left over (the layer
 * takes -1 as another rank's expert). Normalised weights are right where the scores themselves are
 * too small for fp32, too. A sigmoid that is 0 in 64 bits (1 / (1 + exp(-logit)), logits below
 * -709.78) is 0; where all chosen scores are 0 the weights, and their gradients, are 0.
 * logits: fp32 or bf16 [T][E] (logits_dtype); topk_idx: int32 [T][K]; topk_weights: fp32
 * [T][K].
 * Errors: MOE_ERR_INVALID (null or misaligned pointers, T < 0, E not in [1,1024], K not in
 * [1,16] or above the experts of topk_groups groups, groups not in [1,64] or no divisor of
 * E, topk_groups not in [1,groups], group_top not 1 or 2, scale not finite, unknown types).
 */
MOE355_API int moe_router_topk(const void* logits, int32_t logits_dtype, const float* bias, int32_t T, int32_t E,
                               int32_t K, const moe_router_config* cfg, int32_t* topk_idx, float* topk_weights,
                               void* stream);

/*
 * Backward of moe_router_topk: d_logits [T][E] (in logits' type, every element written) from
 * d_topk_weights fp32 [T][K], as moe_combine_backward gives it. The choice itself has no
 * gradient, nor has the bias. topk_idx as moe_router_topk wrote it for these logits; places
 * outside [0, E) or of a switched-off expert count for nothing, an expert that stands in
 * two places counts in both. d_topk_weights is not looked at where topk_idx is -1. logits is
 * read anew: it must hold what it held. d_logits may be logits.
 * Errors: those of moe_router_topk.
 */
MOE355_API int moe_router_topk_backward(const float* d_topk_weights, const void* logits, int32_t logits_dtype,
                                        const int32_t* topk_idx, int32_t T, int32_t E, int32_t K,
                                        const moe_router_config* cfg, void* d_logits, void* stream);

/*
 * moe_dispatch for rows that are quantised already: pool[pos[t,k]] = q[t] with its scale
 * words, moved to their tile-major places. Epoch, workspace, pool_rows, what is left alone and
 * the pool's content are as moe_dispatch with act_dtype has them: with q from moe_rmsnorm the
 * pool has the bits moe_dispatch makes of the bf16 rows (and in MXFP8 zeros in a last scale
 * word's bytes past the row's last block, which nothing reads). A tile's flag is raised, as
 * there, after its rows and scale words are stored, but nearly all of them at the call's end
 * (its workgroups publish once): an FFN that waits for them on another stream begins then.
 * Errors: those of moe_dispatch; MOE_ERR_INVALID for act_dtype MOE_BF16 and misaligned q,
 * q_s or pool.
 */
MOE355_API int moe_dispatch_quantized(const void* q, const void* q_s, int32_t H, int32_t act_dtype,
                                      const moe_plan_t* plan, int32_t pool_rows, void* pool, void* pool_s,
                                      uint32_t epoch, void* ws, size_t ws_bytes, void* stream);

/* Bytes of moe_expert_ffn_decode's workspace: h of every pair with its scales (0 for
 * invalid sizes or T = 0). */
MOE355_API size_t moe_expert_ffn_decode_workspace_bytes(int32_t T, int32_t K, int32_t I);

/*
 * The expert FFN of up to 64 tokens with MXFP4 weights, straight from the routing (no plan,
 * no pool): the layer's mxfp4 mode as matrix-vector products, each reached expert's weights
 * read once:
 *   h[t,k] = silu(W1[e] gate . x[t]) * (W1[e] up . x[t]), quantised to MXFP8;
 *   out[t] = bf16(sum over the local pairs of topk_weights[t,k] * (W2[e] . h[t,k]))
 * with e = topk_idx[t,k] - expert_begin; pairs with e outside [0, E_local) are other ranks'
 * and add nothing, a token without a local pair gets zeros. Products are exact and summed in
 * fp32, in an order that the arguments' shapes and topk_idx fix.
 * x: MXFP8 codes [T][H] with x_s (the quantised rows above; x_dtype MOE_MXFP4), or bf16
 * [T][H] with x_s null (x_dtype MOE_BF16: quantised to MXFP8 on the way, as moe_dispatch
 * does). w1, w2: codes as moe_pack_weights lays them out, w1_s, w2_s: scales as
 * moe_pack_mx_scales does -- what moe_expert_ffn takes in mxfp4 mode. topk_idx: int32 [T][K],
 * topk_weights: fp32 [T][K], out: bf16 [T][H], every row written (bf16 rows of x are held there,
 * quantised, until then). A code times its scale has to be a bf16 number: scale bytes up to 246
 * for x (the largest that bf16 rows get) and 252 for weights, larger values count as infinite;
 * those below 2^-126 are rounded to multiples of 2^-133. Scale byte 255 is NaN.
 * Errors: MOE_ERR_INVALID (null or misaligned pointers, T < 0, K not in [1,16], E_local not
 * in [1,1024], expert_begin < 0, H or I < 1, unknown x_dtype, x_s not as x_dtype wants it,
 * small workspace, out overlapping x), MOE_ERR_UNSUPPORTED (T > 64, H % 128 or I % 128 nonzero, H or I above
 * 32768).
 */
MOE355_API int moe_expert_ffn_decode(const void* x, const void* x_s, int32_t x_dtype, int32_t T, int32_t H, int32_t I,
                                     int32_t K, int32_t expert_begin, int32_t E_local, const int32_t* topk_idx,
                                     const float* topk_weights, const void* w1, const void* w1_s, const void* w2,
                                     const void* w2_s, void* ws, size_t ws_bytes, void* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE355_BLOCK_H */
