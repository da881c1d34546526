/*
 * moe.h — C ABI of libmoe: one GPU's share of an MoE layer, forward and backward,
 * on AMD Instinct MI355X (gfx950).
 *
 * The method is the MoE training path of Ai2's "Introducing Olmo-core 3: open,
 * scalable training infrastructure for large MoE models", section "Scaling and
 * optimizing MoE training": tokens are routed to a few experts, routed rows are
 * written straight into the experts' input buffers (row-wise expert
 * parallelism), routing metadata stays on the GPU so the host never waits for
 * it, the many small expert products run as one grouped GEMM, and MXFP8 can
 * replace BF16 in the expert products.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Every tensor pointer is a DEVICE pointer to caller-owned memory, row-major,
 *    16-byte aligned.  The library never allocates, frees, copies to the host or
 *    synchronises inside these calls; it keeps no per-call state.  Scratch memory
 *    comes from the caller as `ws` of at least the size the matching
 *    *_workspace() function returns (a pure function of the shape).
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).  Every
 *    call only enqueues kernels on it and returns; results are ready when the
 *    stream reaches them.  No device-derived value ever reaches the host.
 *  - Outputs are overwritten (never accumulated into), including zero gradients
 *    for experts that received no rows; the one exception is
 *    moe_router_logits_bwd with accumulate_dx = 1.  Outputs must not alias inputs.
 *  - Errors: arguments are validated on the host before anything is launched.
 *    Invalid values give MOE_EINVAL, valid but unimplemented shapes or types give
 *    MOE_EUNSUPPORTED, a too-small workspace gives MOE_EWORKSPACE; in these
 *    cases nothing is launched.  A failed launch gives MOE_EHIP.  Index arrays
 *    (topk_idx, offsets, perm_*) are trusted: they must come from
 *    moe_route_topk for the same T, E, k.  Non-finite inputs give unspecified
 *    (but memory-safe) results.
 *  - Determinism: identical inputs give identical output bits (no floating-point
 *    atomics; every reduction has a fixed order).
 *
 * Symbols: T tokens, d model width, E experts, k experts per token, f expert
 * hidden width, R = T*k routed rows.  Limits: 1 <= k <= 8, k <= E <= 256,
 * 0 <= T, R < 2^31.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_EINVAL = 1,
  MOE_EUNSUPPORTED = 2,
  MOE_EWORKSPACE = 3,
  MOE_EHIP = 4
} moe_status;

/* Element / compute types.  Data-movement calls take MOE_F32 or MOE_BF16 (the
 * storage type).  The expert FFN takes all three: MOE_F32 (fp32 storage and
 * math), MOE_BF16 (bf16 storage, bf16 MFMA, fp32 accumulate), MOE_MXFP8 (bf16
 * storage and outputs; every expert GEMM runs on MX-scaled FP8 MFMA with
 * operands quantised on the device, fp32 accumulate). */
typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_MXFP8 = 2 } moe_prec;

/* 4: moe_grouped_ffn_bwd takes x_mxt and dy_mxt; the token-axis MX calls. */
int moe_abi_version(void);
const char* moe_status_str(int status);

/* ---------------------------------------------------------------------------
 * Router.
 * ------------------------------------------------------------------------- */

/* Router logits l = x W_r (the routing step of "Scaling and optimizing MoE
 * training"; the pages give no router formula, the plain linear router is used).
 * x [T, d] and w_r [d, E] in `dtype` (MOE_F32 or MOE_BF16); logits [T, E] fp32,
 * fp32 accumulation.  d % 8 == 0. */
int moe_router_logits(const void* x, const void* w_r, int dtype, int64_t T, int32_t d, int32_t E,
                      float* logits, void* stream);

/* Backward of moe_router_logits: dx (+)= dlogits W_r^T and dw_r = x^T dlogits.
 * dlogits [T, E] fp32; dx [T, d] and dw_r [d, E] in `dtype`.  With
 * accumulate_dx = 1 the router term is added to dx (so it joins the output of
 * moe_dispatch_bwd); with 0 dx is overwritten.  dw_r is reduced over tokens in
 * a fixed order through the workspace. */
size_t moe_router_logits_bwd_workspace(int64_t T, int32_t d, int32_t E);
int moe_router_logits_bwd(const void* x, const void* w_r, int dtype, const float* dlogits, int64_t T,
                          int32_t d, int32_t E, void* dx, int accumulate_dx, void* dw_r, void* ws,
                          size_t ws_bytes, void* stream);

/* Top-k routing with the routing metadata built on the device ("Scaling and
 * optimizing MoE training": the metadata stays on the GPU; introduction: four
 * of 8 or 128 experts are chosen per token).
 *   logits [T, E] fp32 (input)
 *   topk_idx [T, k] int32: slot j = j-th expert under (logit descending, index
 *            ascending); -0.0 and +0.0 tie; a NaN logit ranks below every
 *            number (-inf included), NaNs among themselves by index
 *   gates [T, k] fp32: softmax over the k chosen logits (= softmax over all E,
 *            renormalised over the chosen set); NaN for every slot of a token
 *            whose chosen logits include a NaN or whose largest chosen logit
 *            is infinite (a chosen -inf below a finite largest gets gate 0)
 *   counts [E], offsets [E+1] int32: rows per expert and their exclusive prefix
 *            sum (offsets[E] = R)
 *   perm_src [R] int32: expert-buffer row -> flat slot t*k+j (rows of an expert
 *            are in token order)
 *   perm_dst [R] int32: flat slot t*k+j -> expert-buffer row
 *   mx_blk_offsets [E+1] int32 or NULL: prefix sum of ceil(counts/32), the
 *            32-row blocks per expert used by token-axis MX quantisation
 * Bit-exact and deterministic: no atomics decide any order. */
size_t moe_route_topk_workspace(int64_t T, int32_t E, int32_t k);
int moe_route_topk(const float* logits, int64_t T, int32_t E, int32_t k, int32_t* topk_idx,
                   float* gates, int32_t* counts, int32_t* offsets, int32_t* perm_src,
                   int32_t* perm_dst, int32_t* mx_blk_offsets, void* ws, size_t ws_bytes,
                   void* stream);

/* moe_route_topk without a workspace, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid allocation).  Same arguments, outputs and bits as moe_route_topk;
 * the scratch is a static 8 MiB device array that the library holds on each
 * GPU it runs on until the process ends (the current device's copy is used:
 * the stream must belong to the current device).  Limits: T*k <= 2^20 and
 * ceil(T/64)*E <= 2^20, else MOE_EWORKSPACE with nothing launched; MOE_EHIP
 * if the array's device address cannot be obtained.  Every byte of the scratch
 * is written before it is read, so nothing needs clearing between calls, but
 * all calls on one GPU share it: calls that overlap on one GPU (different
 * streams, or host threads) race and give undefined results. */
int moe_route_topk_noalloc(const float* logits, int64_t T, int32_t E, int32_t k, int32_t* topk_idx,
                           float* gates, int32_t* counts, int32_t* offsets, int32_t* perm_src,
                           int32_t* perm_dst, int32_t* mx_blk_offsets, void* stream);

/* Backward of the renormalised gates (the router is trained with the rest of
 * the layer in the MoE training path of "Scaling and optimizing MoE training";
 * the pages give no gradient formula, so this is the exact gradient of the
 * gates moe_route_topk computes): dlogits[t, S_j] = g_j (dg_j - sum_i g_i dg_i),
 * exactly zero for unselected experts (the renormalised gates do not depend on
 * them).  gates, dgates [T, k] fp32, topk_idx [T, k] from moe_route_topk;
 * dlogits [T, E] fp32, overwritten.  MOE_EINVAL / MOE_EUNSUPPORTED for bad
 * sizes or null pointers, nothing launched; T = 0 is a no-op. */
int moe_route_topk_bwd(const float* gates, const float* dgates, const int32_t* topk_idx, int64_t T,
                       int32_t E, int32_t k, float* dlogits, void* stream);

/* Routing by scores (no page gives these formulas; they are the usual ones of
 * layers with many small experts).  A token's scores over the E experts:
 *   MOE_SOFTMAX  s = softmax(logits), MOE_SIGMOID  s = 1 / (1 + exp(-logits))
 * It chooses by c = s + bias (bias [E] fp32, NULL: 0).  `groups` groups of E / groups
 * consecutive experts: a group's worth is the sum of its `group_best` (1 or 2) best
 * choices, and the top_groups worthiest stay in (ties: the lower group).  The k best
 * choices among them, in falling order (ties: the lower index), are topk_idx, and
 *   gates = scale s, or with renorm != 0  scale s / (sum of the k chosen s)
 * (0 where that sum is 0).  The order is that of c in 64 bits, so it does not hang on
 * rounding; gates are rounded once to fp32.  A token of -inf only has scores 0 under
 * softmax; a NaN or +inf logit makes its whole row's scores NaN there; a NaN choice
 * ranks below every number, -inf included, NaNs among themselves by index.
 * counts, offsets, perm_src, perm_dst, mx_blk_offsets (NULL allowed): as
 * moe_route_topk writes them, for the calls that take its metadata.
 * MOE_EINVAL for groups that do not divide E, top_groups outside 1..groups, fewer than
 * k experts in top_groups groups, group_best above a group's size, a scale that is not
 * finite, a null or unaligned pointer; MOE_EUNSUPPORTED for more than 64 groups and for
 * T > 2^28 - 64 (the backward's too).
 * T = 0 is allowed (counts and offsets become zero). */
typedef enum { MOE_SOFTMAX = 0, MOE_SIGMOID = 1 } moe_score;
size_t moe_route_scored_workspace(int64_t T, int32_t E, int32_t k);
int moe_route_scored(const float* logits, const float* bias, int64_t T, int32_t E, int32_t k, int score,
                     int32_t groups, int32_t top_groups, int32_t group_best, int renorm, float scale,
                     int32_t* topk_idx, float* gates, int32_t* counts, int32_t* offsets, int32_t* perm_src,
                     int32_t* perm_dst, int32_t* mx_blk_offsets, void* ws, size_t ws_bytes, void* stream);

/* Backward of moe_route_scored's gates: the gradient of the logits for dgates [T, k]
 * (the choice itself, the groups and the bias have none).  topk_idx [T, k]: distinct
 * experts per token, as moe_route_scored wrote them for these logits; a slot whose
 * index is outside 0..E-1 (a caller's mark of padding) takes no part.  Experts that
 * were not chosen get zero, but under softmax without renorm, where every score
 * depends on all logits.  Under softmax a row with a NaN or +inf logit gives NaN to
 * its chosen experts, as its gates are NaN.  dlogits [T, E] is overwritten, or with accumulate != 0
 * added to (so it joins the gradient of moe_balance_loss_bwd). */
int moe_route_scored_bwd(const float* logits, const int32_t* topk_idx, const float* dgates, int64_t T, int32_t E,
                         int32_t k, int score, int renorm, float scale, int accumulate, float* dlogits, void* stream);

/* Update of the balancing bias from the load of a step: with n[e] the sum over s of
 * counts[s,e] (counts [S, E]: moe_route_scored's with S = 1, or moe_balance_loss's,
 * which leave padded tokens out) bias_out[e] = bias[e] + rate sign(mean(n) - n[e]).
 * bias_out may be bias. */
int moe_route_bias_update(const int32_t* counts, int64_t S, int32_t E, float rate, const float* bias, float* bias_out,
                          void* stream);

/* Load statistics of a routing ("Scaling to the trillion-parameter range":
 * a balance metric alone can be gamed, so the observable load is exported).
 * counts [E] int32 (from moe_route_topk), 1 <= E <= 256; stats [4] int32 on
 * the device, overwritten: {largest expert's rows, smallest expert's rows,
 * number of experts with no rows, total rows}.  MOE_EINVAL for a bad E or a
 * null pointer. */
int moe_route_stats(const int32_t* counts, int32_t E, int32_t* stats, void* stream);

/* Balance loss and z loss of the router, with the per-expert counts
 * ("Scaling to the trillion-parameter range": experts' load is kept even during
 * training; the pages give no formula, these are the usual ones).  With p the
 * softmax of a token's E logits and lse their log-sum-exp, over the tokens that
 * count in sequence s (n_s of them; S' sequences have any; N = sum n_s):
 *   counts[s,e] = chosen slots of expert e, probs[s,e] = mean of p[e] (0 if n_s = 0)
 *   loss[0] = alpha / S' sum_s E sum_e counts[s,e] / (k n_s) probs[s,e]
 *   loss[1] = zeta / N sum_t lse_t^2                         (both 0 if N = 0)
 *   lse [T]: 0 for a token that does not count
 *   norm [S + 2] fp32: S', N, then n_s (rounded past 2^24), kept for the backward
 * seq_offsets [S+1] int32 (device, non-decreasing, within [0, T]): sequence s
 * holds tokens [seq_offsets[s], seq_offsets[s+1]); empty sequences are allowed,
 * and tokens before the first or behind the last one do not count.  NULL (then
 * S = 1): one sequence of all T tokens.  A token counts when it is in a sequence,
 * token_mask [T] (uint8, NULL: all) is nonzero and some logit is above -inf (a
 * token of -inf only chooses nothing).  A counted token with a NaN or +inf logit
 * makes the losses NaN; what masked tokens hold does not matter.
 * topk_idx [T, k] from moe_route_topk; logits [T, E] fp32; counts [S, E] int32;
 * probs [S, E], lse, loss [2] fp32.  Sums are
 * fp32 over at most 32 tokens and fp64 beyond, in a fixed order.
 * The backward writes
 *   dlogits[t,e] = p_e (a_e - sum_j a_j p_j) + dloss[1] 2 zeta / N lse_t p_e,
 *   a_e = dloss[0] alpha E counts[s,e] / (k n_s^2 S')       (no gradient through counts)
 * and zero for tokens that do not count, whatever dloss holds; with gates and dgates (both or
 * neither; then topk_idx too) the gates' gradient of moe_route_topk_bwd is
 * added for every token in the same pass, so that call is not needed.
 * dloss [2] fp32 on the device: upstream gradients of the two losses (NULL: 1).
 * Errors as for moe_route_topk; MOE_EINVAL also for a non-finite alpha or zeta,
 * S < 1, and S > 1 without seq_offsets, MOE_EUNSUPPORTED for T > 2^29 - 32.  T = 0 is allowed (losses 0). */
size_t moe_balance_loss_workspace(int64_t T, int32_t E, int64_t S);
int moe_balance_loss(const float* logits, const int32_t* topk_idx, int64_t T, int32_t E, int32_t k,
                     const int32_t* seq_offsets, int64_t S, const uint8_t* token_mask, float alpha, float zeta,
                     float* loss, int32_t* counts, float* probs, float* lse, float* norm, void* ws,
                     size_t ws_bytes, void* stream);
int moe_balance_loss_bwd(const float* logits, const float* lse, const int32_t* counts, const float* norm, int64_t T,
                         int32_t E, int32_t k, const int32_t* seq_offsets, int64_t S, const uint8_t* token_mask,
                         float alpha, float zeta, const float* dloss, const int32_t* topk_idx, const float* gates,
                         const float* dgates, float* dlogits, void* stream);

/* ---------------------------------------------------------------------------
 * Layer norm of the token rows, the norm before the router and the experts (no
 * page defines it; the usual formula).  x [T, d] in `dtype` (MOE_F32 or
 * MOE_BF16), any d from 1 to 2^20.
 *   forward:  s = x, or x + residual rounded to `dtype` (stored in `sum` unless
 *             NULL; sum without residual is MOE_EINVAL);
 *             mean, rstd = 1 / sqrt(var + eps) of each row of s, fp32 [T] (each
 *             may be NULL); y = (s - mean) rstd weight + bias
 *   backward: of y for upstream dy, with x the rows that were normalised (s):
 *             dx = rstd (v - avg(v) - h avg(v h)) (+ dres), v = dy weight,
 *             h = (x - mean) rstd; dw = sum_t dy h, db = sum_t dy
 * weight, bias, residual, dres, dw, db may be NULL (weight 1, bias 0, none);
 * weight, bias, dw, db [d] in `dtype`.  dres [T, d] is a gradient that reaches
 * s by another way (the residual stream's).  Statistics and sums are fp32.
 * A constant row with eps = 0 gives NaN.  In place: y or sum may be x or residual,
 * dx may be dy, x or dres; no other overlap.  T = 0 is allowed: dw and db become
 * zero.  The workspace is needed for dw and db only.  MOE_EINVAL for d < 1 and for
 * an eps that is negative or not finite, MOE_EUNSUPPORTED for d > 2^20. */
int moe_layernorm(const void* x, const void* residual, const void* weight, const void* bias, int dtype, int64_t T,
                  int32_t d, float eps, void* y, void* sum, float* mean, float* rstd, void* stream);
size_t moe_layernorm_bwd_workspace(int64_t T, int32_t d);
int moe_layernorm_bwd(const void* dy, const void* x, const void* weight, const float* mean, const float* rstd,
                      const void* dres, int dtype, int64_t T, int32_t d, void* dx, void* dw, void* db, void* ws,
                      size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Row-wise dispatch and weighted combine ("Scaling and optimizing MoE
 * training": routed data goes directly into the experts' input buffers).
 * All in `dtype` (MOE_F32 or MOE_BF16), d % 8 == 0.
 * ------------------------------------------------------------------------- */

/* x_perm[perm_dst[t*k+j]] = x[t]: each token row is read once and written to
 * its k rows of the expert-major buffer.  x [T, d], x_perm [R, d]; exact copy. */
int moe_dispatch(const void* x, int dtype, int64_t T, int32_t d, int32_t k, const int32_t* perm_dst,
                 void* x_perm, void* stream);

/* dx[t] = sum_j dx_perm[perm_dst[t*k+j]] (fp32 sum in slot order). */
int moe_dispatch_bwd(const void* dx_perm, int dtype, int64_t T, int32_t d, int32_t k,
                     const int32_t* perm_dst, void* dx, void* stream);

/* out[t] = sum_j gates[t,j] * y_perm[perm_dst[t*k+j]] (fp32 sum in slot order).
 * y_perm [R, d] holds the unweighted expert outputs; out [T, d]. */
int moe_combine(const void* y_perm, int dtype, const float* gates, const int32_t* perm_dst,
                int64_t T, int32_t d, int32_t k, void* out, void* stream);

/* Backward of moe_combine for upstream gradient dout [T, d]:
 *   dy_perm[perm_dst[t*k+j]] = gates[t,j] * dout[t]          ([R, d], dtype)
 *   dgates[t,j] = <dout[t], y_perm[perm_dst[t*k+j]]>          ([T, k], fp32) */
int moe_combine_bwd(const void* dout, const void* y_perm, int dtype, const float* gates,
                    const int32_t* perm_dst, int64_t T, int32_t d, int32_t k, void* dy_perm,
                    float* dgates, void* stream);

/* MXFP8 data movement ("Scaling and optimizing MoE training": the MXFP8 gains
 * came from the expert FFN and from moving data between experts): the two
 * calls that write an expert-major buffer the MXFP8 FFN quantises along d
 * (X for the gate/up GEMM, dY for the down-projection's data gradient) also
 * write its MX rows layout, so the FFN skips that quantisation pass.
 * The MX buffer `*_mx` (caller-owned, moe_mx_act_bytes(R, d) bytes, R = T*k)
 * holds the E4M3 codes [R, d] (blocks of 32 along d, as mx_quantize axis 1),
 * then, at the next 256-byte boundary, the E8M0 bytes in grouped order: the
 * byte of (row r, block b) at ((b/4)*R + r)*4 + b%4.  Codes and scales are
 * bit-identical to mx_quantize of the bf16 buffer the same call writes.
 * bf16 only; d % 128 == 0 (else MOE_EUNSUPPORTED); otherwise as moe_dispatch /
 * moe_combine_bwd.  moe_mx_act_bytes returns 0 for invalid sizes. */
size_t moe_mx_act_bytes(int64_t rows, int32_t cols);
int moe_dispatch_mx(const void* x, int64_t T, int32_t d, int32_t k, const int32_t* perm_dst,
                    void* x_perm, void* x_mx, void* stream);
int moe_combine_bwd_mx(const void* dout, const void* y_perm, const float* gates, const int32_t* perm_dst,
                       int64_t T, int32_t d, int32_t k, void* dy_perm, float* dgates, void* dy_mx,
                       void* stream);

/* MXFP8 data movement with the token-axis layout ("Scaling and optimizing MoE
 * training": the MXFP8 gains came from the expert FFN and from moving data
 * between experts).  The weight gradients contract over each expert's tokens,
 * so the MXFP8 backward needs X and dY also quantised along the tokens, per
 * expert segment; these two calls write that layout together with the rows
 * layout of moe_dispatch_mx / moe_combine_bwd_mx, from one destination-major
 * pass that reads each expert row's token row directly, so the bf16 expert rows
 * need not be written at all (x_perm / dy_perm may be NULL; given, they receive
 * the same rows as moe_dispatch / moe_combine_bwd).
 * Token-axis layout of an expert-major [R, cols] buffer (the MX buffer `*_mxt`,
 * caller-owned, moe_mx_tok_bytes(R, E, cols) bytes): Rp = moe_mx_tok_rows(R, E)
 * padded token positions, expert e's 32-row blocks at positions
 * [32 mx_blk_offsets[e], 32 mx_blk_offsets[e+1]) (mx_blk_offsets from
 * moe_route_topk; a segment's last block zero-padded, positions past the last
 * segment zero); E4M3 codes [cols, Rp] (column c, position p at c Rp + p), then
 * at the next 256-byte boundary the E8M0 bytes, the byte of (column c, block b)
 * at ((b/4) cols + c) 4 + b%4.  Codes and scales are bit-identical to
 * mx_quantize(axis 0, seg_offsets = offsets) of the bf16 expert rows (scales
 * regrouped as stated).  The rows layout `*_mx` is as for moe_dispatch_mx.
 * moe_combine_bwd_mx_tok also writes dgates (as moe_combine_bwd); dY = gate x
 * dout is rounded to bf16 before it is encoded, as moe_combine_bwd stores it.
 * perm_src, offsets, mx_blk_offsets: from moe_route_topk for the same T, E, k.
 * bf16 only; d % 128 == 0 (else MOE_EUNSUPPORTED); 1 <= E <= 256; otherwise as
 * moe_dispatch / moe_combine_bwd.  moe_mx_tok_rows / _bytes return 0 for
 * invalid sizes. */
int64_t moe_mx_tok_rows(int64_t R, int32_t E);
size_t moe_mx_tok_bytes(int64_t R, int32_t E, int32_t cols);
int moe_dispatch_mx_tok(const void* x, int64_t T, int32_t d, int32_t k, int32_t E, const int32_t* perm_src,
                        const int32_t* offsets, const int32_t* mx_blk_offsets, void* x_perm, void* x_mx,
                        void* x_mxt, void* stream);
int moe_combine_bwd_mx_tok(const void* dout, const void* y_perm, const float* gates, const int32_t* perm_dst,
                           const int32_t* perm_src, const int32_t* offsets, const int32_t* mx_blk_offsets,
                           int64_t T, int32_t d, int32_t k, int32_t E, void* dy_perm, float* dgates, void* dy_mx,
                           void* dy_mxt, void* stream);

/* ---------------------------------------------------------------------------
 * Grouped SwiGLU expert FFN ("Scaling and optimizing MoE training": the small
 * per-expert products run as one grouped GEMM; MXFP8 where it pays).
 * Rows of expert e are [offsets[e], offsets[e+1]) of the expert-major buffer
 * (device metadata from moe_route_topk; the host never reads it).
 *   w_gate, w_up [E, d, f], w_down [E, f, d]   (x @ W orientation)
 *   forward:  h_gate = X We_g, h_up = X We_u, a_act = silu(h_gate) * h_up,
 *             y_perm = a_act We_d  (unweighted; the gate is applied in combine)
 *   backward: dA = dY Wd^T, dh_up = dA silu(Hg), dh_gate = dA Hu s (1 + Hg (1 - s)),
 *             dx_perm = dh_gate Wg^T + dh_up Wu^T,
 *             dw_down = A^T dY, dw_gate = X^T dh_gate, dw_up = X^T dh_up
 *             (all experts written; zero for experts with no rows)
 * Storage: fp32 for MOE_F32, bf16 for MOE_BF16 and MOE_MXFP8.  h_gate, h_up,
 * a_act [R, f] are saved by the forward and read by the backward.
 * MOE_MXFP8 quantises every GEMM operand on the device to E4M3 with one E8M0
 * scale per 32 elements along that GEMM's contraction axis (as mx_quantize).
 * Limits: d % 64 == 0 and f % 64 == 0 (MOE_MXFP8: % 128).  mx_blk_offsets
 * (from moe_route_topk) is required by the MOE_MXFP8 backward, else ignored.
 * mx_wcache (MOE_MXFP8 only, else ignored; may be NULL): a cache built by
 * moe_mx_weight_cache_build from these same weights, E, d and f; with it the
 * call quantises no weight (w_gate/w_up/w_down are still passed and
 * validated); results are bit-identical to those without it.
 * x_mx (forward) / dy_mx (backward) (MOE_MXFP8 only, else MOE_EINVAL; may be
 * NULL): x_perm / dy_perm already in the MX rows layout written by
 * moe_dispatch_mx / moe_combine_bwd_mx (or the _tok calls) for the same buffer;
 * the call then does not quantise it again (bit-identical results).
 * x_mxt / dy_mxt (backward, MOE_MXFP8 only, else MOE_EINVAL; may be NULL): X / dY
 * in the token-axis layout of moe_dispatch_mx_tok / moe_combine_bwd_mx_tok, used
 * by the weight gradients instead of quantising x_perm / dy_perm along the
 * tokens (bit-identical results).  With MOE_MXFP8, x_perm may be NULL when the
 * forward has x_mx and the backward x_mxt, and dy_perm when the backward has
 * both dy_mx and dy_mxt. */
size_t moe_grouped_ffn_workspace(int64_t R, int32_t E, int32_t d, int32_t f, int prec, int is_bwd);
int moe_grouped_ffn_fwd(int64_t R, int32_t E, int32_t d, int32_t f, int prec, const int32_t* offsets,
                        const void* x_perm, const void* w_gate, const void* w_up, const void* w_down,
                        const void* mx_wcache, const void* x_mx, void* h_gate, void* h_up, void* a_act,
                        void* y_perm, void* ws, size_t ws_bytes, void* stream);
int moe_grouped_ffn_bwd(int64_t R, int32_t E, int32_t d, int32_t f, int prec, const int32_t* offsets,
                        const int32_t* mx_blk_offsets, const void* dy_perm, const void* x_perm,
                        const void* h_gate, const void* h_up, const void* a_act, const void* w_gate,
                        const void* w_up, const void* w_down, const void* mx_wcache, const void* dy_mx,
                        const void* x_mxt, const void* dy_mxt, void* dx_perm, void* dw_gate, void* dw_up,
                        void* dw_down, void* ws, size_t ws_bytes, void* stream);

/* Pre-quantised MXFP8 expert weights ("Scaling and optimizing MoE training":
 * converting into MXFP8 has a cost the savings must exceed).  Weights change
 * once per optimiser step, so a loop with several micro-batches per step can
 * quantise them once: the cache holds each of w_gate, w_up [E, d, f] and
 * w_down [E, f, d] (bf16) in both orientations the MXFP8 FFN uses (forward:
 * blocks along d for w_gate/w_up and along f for w_down; backward: blocks along
 * the last axis), each produced from a single read of the weight.
 * moe_mx_weight_cache_bytes(E, d, f) = 6 E d f (1 + 1/32) bytes plus alignment.
 * Layout (the FFN calls take the cache back unchanged; it is stated so that it
 * can be inspected or stored): six regions in the order w_gate, w_up, w_down
 * forward, then w_gate, w_up, w_down backward; each region is its E4M3 codes
 * (E d f bytes) and then its E8M0 scale bytes (E d f / 32), both parts starting
 * on a 256-byte boundary.  A forward region holds each expert's weight
 * quantised down its rows and stored transposed ([E, f, d] for w_gate/w_up,
 * [E, d, f] for w_down; blocks run along the last axis); with M the rows and
 * K the last axis of that stored form, the scale of expert e, row m, block b
 * is byte e M (K/32) + ((b/4) M + m) 4 + b%4.  A backward region keeps the
 * weight's own shape with blocks along its last axis, and the scale of expert
 * e, row m, block b is byte ((b/4) E M + e M + m) 4 + b%4.  The cache stays
 * valid while the weights are unchanged; building
 * again overwrites it.  Errors: MOE_EINVAL (null or unaligned pointer, bad E,
 * d, f), MOE_EUNSUPPORTED (d or f not a multiple of 128), MOE_EWORKSPACE
 * (cache_bytes too small); nothing is launched then. */
size_t moe_mx_weight_cache_bytes(int32_t E, int32_t d, int32_t f);
int moe_mx_weight_cache_build(const void* w_gate, const void* w_up, const void* w_down, int32_t E,
                              int32_t d, int32_t f, void* cache, size_t cache_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * MXFP8 quantiser ("Scaling and optimizing MoE training" names MXFP8 and the
 * cost of converting into it; the format follows the public OCP MX v1.0 spec):
 * blocks of 32 consecutive elements along `axis`; scale exponent
 * e = floor(log2(max|v|)) - 8 clamped to [-127, 127] (all-zero block: -127),
 * stored as the E8M0 byte e + 127; elements v / 2^e rounded to nearest-even
 * E4M3 (bias 7), saturated to +-448, sign kept.
 *   src [batch, rows, cols] in src_dtype (MOE_F32 or MOE_BF16).
 *   axis 1: q [batch, rows, cols], scales [batch, rows, cols/32]; cols % 32 == 0.
 *   axis 0, seg_offsets NULL: blocks run down the rows and are stored
 *           contiguously, i.e. transposed: q [batch, cols, rows],
 *           scales [batch, cols, rows/32]; rows % 32 == 0.
 *   axis 0 with seg_offsets (device int32, nseg+1 prefix offsets of row
 *           segments, seg_offsets[nseg] = rows, 1 <= nseg <= 256; batch == 1):
 *           blocks restart at
 *           each segment and a segment's last block is zero-padded.  With
 *           B_s = sum_{s'<s} ceil(n_s'/32) and Rp = 32*(ceil(rows/32) + nseg),
 *           q is [cols, Rp] with segment s in columns [32 B_s, 32 B_{s+1}),
 *           scales [cols, Rp/32]; columns past 32 B_nseg are written as zero
 *           codes with scale byte 0.
 * cols % 8 == 0 for axis 0. */
int mx_quantize(const void* src, int src_dtype, int64_t batch, int64_t rows, int64_t cols,
                int32_t axis, const int32_t* seg_offsets, int32_t nseg, uint8_t* q,
                uint8_t* scales, void* stream);

/* ---------------------------------------------------------------------------
 * Orthogonalised updates of the expert weights (no page gives an optimiser
 * formula; Newton-Schulz orthogonalisation as in the published Muon optimiser).
 * For each of E matrices U [rows, cols] on its own:
 *   X = U / (|U|_F + eps);  `steps` times:  X <- a X + (b A + c A^2) X, A = X X^T
 * moe_orthogonalize: U = g; out = X.
 * moe_muon_step:     mom_out = momentum mom + g (fp32);
 *                    U = g + momentum mom_out (nesterov != 0) or mom_out;
 *                    w_out = (1 - lr weight_decay) w - lr scale X.
 * g, out, w, w_out [E, rows, cols] in `dtype` (MOE_F32 or MOE_BF16); mom, mom_out
 * [E, rows, cols] fp32.  mom_out may be mom and w_out may be w (in place); no other
 * overlap.  coef: HOST array [steps][3] of a, b, c, read before the call returns;
 * NULL: 3.4445, -4.7750, 2.0315 in every step.
 * Accuracy: fp32 sums; products on matrix cores, with operands of 22 mantissa bits
 * for MOE_F32, and of 11 for MOE_BF16, where the a X term takes X with 15 (matrices
 * of one workgroup: 22) in all steps but the last.  With the default coefficients
 * that is 0.08 to 0.15% (rms) beside the 0.17% of the result's rounding to bf16.  A
 * zero matrix gives zeros; a non-finite element makes its own matrix NaN only.
 * Limits: rows, cols <= 32768 with rows x cols (rounded up to 64) < 2^30,
 * E <= 65535, 1 <= steps <= 16, and coefficients whose polynomial keeps singular
 * values and its own terms within 15 over all steps (fp16 operands), else
 * MOE_EUNSUPPORTED; MOE_EINVAL for non-finite scalars (lr scale and lr weight_decay
 * among them) and negative eps.  E = 0 is a no-op.  One workspace size serves both
 * calls. */
size_t moe_orthogonalize_workspace(int32_t E, int32_t rows, int32_t cols, int dtype);
int moe_orthogonalize(const void* g, int dtype, int32_t E, int32_t rows, int32_t cols, int32_t steps,
                      const float* coef, float eps, void* out, void* ws, size_t ws_bytes, void* stream);
int moe_muon_step(const void* g, int dtype, int32_t E, int32_t rows, int32_t cols, const float* mom, float momentum,
                  int nesterov, int32_t steps, const float* coef, float eps, const void* w, float lr,
                  float weight_decay, float scale, float* mom_out, void* w_out, void* ws, size_t ws_bytes,
                  void* stream);

/* ---------------------------------------------------------------------------
 * Dense product with bias, activation and residual (a shared expert beside the
 * routed ones; no page defines it).  In `dtype` (MOE_F32 or MOE_BF16), fp32 sums,
 * each output rounded once:
 *   forward:  z = x w + bias, y = act(z) + residual
 *   backward: dz = dy act'(z), dx = (dz w^T) in_act'(in_z) + dres, dw = x^T dz,
 *             db = sum of dz over the rows
 * x, dx, in_z, dres [M, K]; w, dw [K, N]; y, dy, z, residual [M, N]; bias, db [N]; any
 * sizes (K, N up to 2^20).  bias, residual, z (forward: not kept) and dres may be NULL, and so
 * may any of dx, dw, db (not computed).  The backward takes z as the forward kept it;
 * with act MOE_ACT_NONE it needs none.  in_z, in_act: the pre-activation and activation
 * that x came from, so that dx is the gradient of that in_z; MOE_ACT_NONE: dx is that of x.
 * MOE_ACT_GELU is z Phi(z) with the error function; relu'(0) = 0.  For MOE_BF16 the products
 * take dz rounded to bf16 (db does not).  y may be residual; dx may be dres or in_z; no
 * other overlap.  M = 0 is allowed (dw and db become zero).  MOE_EUNSUPPORTED for K or N
 * past 2^20, for more than 2^35 elements (rounded up to 8 columns), and for rows of few columns
 * from about 2^30 (fp32) or 2^31 (bf16) on, whose launch would hold 2^32 threads. */
typedef enum { MOE_ACT_NONE = 0, MOE_ACT_RELU = 1, MOE_ACT_SILU = 2, MOE_ACT_GELU = 3 } moe_act;
size_t moe_linear_workspace(int dtype, int64_t M, int32_t K, int32_t N, int is_bwd);
int moe_linear(const void* x, const void* w, const void* bias, const void* residual, int dtype, int64_t M, int32_t K,
               int32_t N, int act, void* y, void* z, void* ws, size_t ws_bytes, void* stream);
int moe_linear_bwd(const void* dy, const void* x, const void* w, const void* z, int dtype, int64_t M, int32_t K,
                   int32_t N, int act, const void* in_z, int in_act, const void* dres, void* dx, void* dw, void* db,
                   void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * AdamW step of a list of tensors (no page gives an optimiser formula; AdamW as
 * published).  With g times *grad_scale (device, NULL: 1) and t the step:
 *   m' = beta1 m + (1 - beta1) g,  v' = beta2 v + (1 - beta2) g^2
 *   w' = (1 - r weight_decay) w - r m' / (1 - beta1^t) / (sqrt(v' / (1 - beta2^t)) + eps)
 * with r = lr lr_scale, in fp32.  `tensors` is a HOST array, read before the call returns;
 * w, g, w_out of a tensor in `dtype` (MOE_F32 or MOE_BF16), w_out may be w.
 * The states of all tensors lie in one buffer each, a tensor's at elements
 * [offset, offset + n) with offset a multiple of 32, rising over the list without overlap;
 * what follows up to the next multiple of 32 belongs to it and stays zero.
 *   bits 32: m, v fp32 [state_len]
 *   bits 8:  m and the root of v as E4M3 codes [state_len] with one byte b per 32 values
 *            ([state_len / 32], it stands for 2^(b - 127); 255: a value was not finite, the
 *            block reads as NaN).  The power of two is the least that keeps the block's
 *            largest value within 448.  A value between two codes takes the upper one if
 *            its place between them and a random number in (0, 1) sum to 1 or more: the number
 *            is (r + 1/2) / 2^16 with r the high (m) or low (root of v) half of
 *            hash(i 0x9E3779B9 + hash(hash(seed + j 0x9E3779B9) + t 0x9E3779B9)) for
 *            element i of tensor j, all modulo 2^32.  A root above 0 is at least the least code.
 *            (Values below 2^-126 are taken as fp32 has them there, a root above 0 above 0.)
 * master (MOE_BF16 only, NULL: none): fp32 weights [state_len]; the step is theirs, and
 * w_out their rounding (w is not read).  All *_out buffers may be their inputs; no other
 * overlap, and no tensor twice.
 * step_dev (NULL: `step` counts): t on the device, at least 1, for captured graphs.
 * MOE_EINVAL for betas outside [0, 1), an eps that is neither 0 nor within 2^-126 .. 2^100,
 * scalars that are not finite (products of lr, lr_scale and weight_decay among them), step < 1,
 * n < 0 (0 is skipped), bad offsets, a null or unaligned pointer, a master with MOE_F32;
 * MOE_EUNSUPPORTED for 2^37 elements or more in a tensor.  A launch takes 56 tensors. */
typedef struct {
  const void* w;
  const void* g;
  void* w_out;
  int64_t n;
  int64_t offset;
  float weight_decay;
  float lr_scale;
} moe_adamw_tensor;
int moe_adamw_step(const moe_adamw_tensor* tensors, int32_t count, int dtype, int bits, int64_t state_len,
                   const void* m, const void* v, const uint8_t* m_scale, const uint8_t* v_scale, const float* master,
                   double lr, double beta1, double beta2, double eps, int64_t step, const int64_t* step_dev,
                   const float* grad_scale, uint32_t seed, void* m_out, void* v_out, uint8_t* m_scale_out,
                   uint8_t* v_scale_out, float* master_out, void* stream);

/* The values of 8-bit states (m and the root of v, as moe_adamw_step keeps them) in bf16 [state_len],
 * which holds them exactly (scales below 2^-124 apart). */
int moe_adamw_state_values(const uint8_t* m, const uint8_t* m_scale, const uint8_t* v, const uint8_t* v_scale,
                           int64_t state_len, void* m_values, void* root_values, void* stream);

/* ---------------------------------------------------------------------------
 * Diagnostics: per-kernel timing for benchmarks and profiling (no page
 * defines it).  While enabled, every kernel the library launches is bracketed
 * by two HIP events recorded on the caller's stream; events come from a pool
 * that grows on first use, so enable it and run one warm-up pass before a timed
 * region.  moe_timing_enable(1) also discards earlier records; (0) stops.
 * moe_timing_report waits for the recorded events and writes one text line per
 * kernel name, "<name> <launches> <total_ms>\n", NUL-terminated, into buf
 * (MOE_EINVAL if len is too small), then discards the records.  Process-wide
 * state guarded by a mutex.
 * ------------------------------------------------------------------------- */
int moe_timing_enable(int on);
int moe_timing_report(char* buf, size_t len);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H */
