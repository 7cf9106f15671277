/*
 * epdc_router.h - what runs before the dispatch of an MoE layer on one MI355X
 * (gfx950).
 *
 * Third header of libepdc.so: from the residual stream to the inputs of
 * epdc.h.  The RMS norm with the residual's addition and an output in 8 bits,
 * the router's logits, the choice of the experts, the gradients of all three,
 * and the dispatch of rows that are in 8 bits already.
 *
 * The conventions are those of epdc.h: device pointers to row-major,
 * contiguous arrays; the caller owns every buffer; the library allocates
 * nothing, keeps no state and never synchronizes; a call validates its
 * arguments on the host, returns a negative ep_status_t before anything is
 * enqueued if one is bad, and otherwise only enqueues kernels on `stream`.
 * The arrays belong to the current device.  A pointer to an empty array may
 * be NULL.  Outputs must not overlap inputs unless a call says so.  No result
 * depends on the order in which workgroups run.
 */
#ifndef EPDC_ROUTER_H
#define EPDC_ROUTER_H

#include "epdc.h"

#ifdef __cplusplus
extern "C" {
#endif

#define EPDC_ROUTER_ABI_VERSION 1
/* Channels of a row of the norm, and of the router. */
#define EPDC_NORM_CHANNELS 32768
#define EPDC_ROUTER_CHANNELS 65536
/* Groups of experts ep_route chooses from. */
#define EPDC_MAX_GROUPS 16

/* Version of this header's ABI (EPDC_ROUTER_ABI_VERSION). */
int ep_router_abi_version(void);

/* Types of the norm's weight. */
typedef enum { EP_NORM_W_BF16 = 0, EP_NORM_W_F32 = 1 } ep_norm_weight_t;

/*
 * RMS norm, after the residual's addition where there is one:
 *   s[t,:]  = bf16( x[t,:] + residual[t,:] )        (fp32 sum; s = x without)
 *   rstd[t] = 1 / sqrt( mean(s[t,:]^2) + eps )
 *   y[t,h]  = s[t,h] * rstd[t] * weight[h]
 *   out     = bf16(fp32(y))
 *   q, scale: e4m3 codes and one scale per 128 channels of y, not of out: amax =
 *             max |y|, scale = fp32(amax / 448), or the smallest power of two at or
 *             above that, code = e4m3(fp32(y / scale)).
 * rstd is in 64 bits, from fp32 sums of the squares of two neighbours, or from 64-bit
 * squares where fp32 does not hold the row's (below 2^-100 with H * eps, or past its
 * largest); y is in 64 bits where there are codes, in fp32 without.  The rstd that is
 * written is infinite where fp32 cannot hold it: rows whose root mean square lies below
 * 2^-128, with an eps as small.
 * The rounding of the codes, saturation, zeros, NaN and infinities follow
 * ep_dispatch_permute's fp8 form.  A group whose scale is 0 (amax below
 * 448 * 2^-150) has codes 0.
 *
 *   x             [T,H] bf16 in (16-byte aligned)
 *   residual      [T,H] bf16 in, or NULL (16-byte aligned)
 *   weight        [H] bf16 or fp32 in, by weight_type (16-byte aligned)
 *   eps           >= 0, finite.  With 0 a row of zeros gives NaN
 *   residual_out  [T,H] bf16 out: s (16-byte aligned); needed with a residual,
 *                 NULL without one.  It may be the residual or x itself
 *   out           [T,H] bf16 out, or NULL (16-byte aligned)
 *   q             [T,H] e4m3 codes out, or NULL (16-byte aligned; H then is a
 *                 multiple of 128); scale [T,H/128] fp32 out, NULL with q
 *   scale_fmt     EP_SCALE_F32 or EP_SCALE_POW2
 *   rstd          [T] fp32 out, or NULL: ep_rms_norm_backward takes it
 * H is a multiple of 8, <= EPDC_NORM_CHANNELS.  One of out and q is given.
 */
int ep_rms_norm(const void* x, const void* residual, const void* weight, int weight_type,
                int64_t num_tokens, int hidden, float eps, void* residual_out, void* out, void* q,
                float* scale, int scale_fmt, float* rstd, hipStream_t stream);

/*
 * Bytes of workspace ep_rms_norm_backward needs for the weight's gradient; 0
 * for sizes it rejects.  Nothing in it has to be cleared, and nothing is kept
 * in it from one call to the next.  Calls that may overlap in time must use
 * different workspaces.
 */
size_t ep_rms_norm_backward_workspace_bytes(int64_t num_tokens, int hidden);

/*
 * Gradient of ep_rms_norm.  With n = s * rstd and g = dy * weight (fp32),
 *   dx[t,:]    = bf16( rstd * (g - n * mean(g * n)) + d_residual[t,:] )
 *   dweight[h] = sum over t of dy[t,h] * n[t,h]     (fp32)
 * dx is the gradient of x and of the residual alike.  The gradient passes the
 * 8-bit output's rounding as if there were none.  A row whose rstd is infinite has NaN.
 *
 *   dy          [T,H] bf16 in: the gradient of y (16-byte aligned)
 *   s           [T,H] bf16 in: residual_out, or x without a residual
 *   weight      as above; rstd [T] fp32 in: of the forward
 *   d_residual  [T,H] bf16 in, or NULL: the gradient that reaches residual_out
 *               from elsewhere.  dx may be d_residual itself, or dy
 *   dx          [T,H] bf16 out (16-byte aligned)
 *   dweight     [H] fp32 out, or NULL
 *   workspace   256-byte aligned; may be NULL (and workspace_bytes 0) when
 *               dweight is
 */
int ep_rms_norm_backward(const void* dy, const void* s, const void* weight, int weight_type,
                         const float* rstd, const void* d_residual, int64_t num_tokens, int hidden,
                         void* dx, float* dweight, void* workspace, size_t workspace_bytes,
                         hipStream_t stream);

/*
 * Bytes of workspace ep_router_logits and ep_router_logits_backward need; 0
 * for sizes they reject.  The rules of the norm's workspace hold.
 */
size_t ep_router_logits_workspace_bytes(int64_t num_tokens, int num_experts, int hidden);
size_t ep_router_logits_backward_workspace_bytes(int64_t num_tokens, int num_experts, int hidden);

/*
 * The router's logits in fp32 from bf16 rows and weights:
 *   logits[t,e] = sum over h of x[t,h] * w[e,h],
 * products exact, sums in fp32.
 *
 *   x          [T,H] bf16 in (16-byte aligned)
 *   w          [E,H] bf16 in (16-byte aligned)
 *   logits     [T,E] fp32 out
 *   workspace  256-byte aligned
 * H is a multiple of 8, <= EPDC_ROUTER_CHANNELS; E <= EPDC_MAX_BINS.
 */
int ep_router_logits(const void* x, const void* w, int64_t num_tokens, int num_experts, int hidden,
                     float* logits, void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Gradient of ep_router_logits:
 *   dx[t,h] = bf16( sum over e of dlogits[t,e] * w[e,h] )
 *   dw[e,h] = sum over t of dlogits[t,e] * x[t,h]   (fp32)
 * dlogits takes part as the sum of bf16 numbers: of two for dx (off by at most
 * 2^-16 of it, beside the 2^-8 of dx's rounding), of three for dw (off by at
 * most 2^-24).  The parts are exact down to the least bf16 number: an entry
 * below 2^-109 in magnitude is off by up to 2^-133 besides.  Where an x or w
 * is infinite, a sum that it enters comes out as NaN or infinite, whichever
 * the formula gives, since one of the parts it meets may be 0.
 *
 *   dlogits    [T,E] fp32 in
 *   x, w       as above; x may be NULL when dw is, w when dx is
 *   dx         [T,H] bf16 out, or NULL (16-byte aligned)
 *   dw         [E,H] fp32 out, or NULL (16-byte aligned)
 *   workspace  256-byte aligned
 */
int ep_router_logits_backward(const float* dlogits, const void* x, const void* w,
                              int64_t num_tokens, int num_experts, int hidden, void* dx, float* dw,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Scores of ep_route. */
typedef enum { EP_SCORE_SOFTMAX = 0, EP_SCORE_SIGMOID = 1 } ep_score_t;

/*
 * The choice of a token's experts from its logits l:
 *   s[e]    = softmax(l)[e] over all E experts, or 1 / (1 + exp(-l[e]))
 *   key[e]  = s[e] + bias[e]     (s[e] without a bias)
 *   groups: the E / num_groups experts from g * E / num_groups on are group g.
 *           A group's worth is the sum of its group_top largest keys; the
 *           topk_groups worthiest groups stay
 *   topk_idx[t,0..K) = the experts of the K largest keys in the groups that
 *           stay, the largest first
 *   topk_weights[t,k] = scale * s[e_k], divided by the sum of the chosen
 *           experts' s where `renormalize` is set (0 where that sum is 0)
 * Scores, keys and weights are computed in 64 bits and a weight is rounded
 * once to fp32.  Keys that agree in their first 42 bits count as equal (43
 * significant bits, the last cut off), and so do worths that agree to 2^-40;
 * the lowest index wins.  All groups staying (topk_groups == num_groups) is one
 * group.  Without a bias, and with one group or group_top 1, the logits themselves
 * are compared, which orders alike, and exactly.
 *
 * An expert is not chosen where its logit is NaN or -infinity, or its key is.
 * A slot that finds no expert has id -1 and weight 0, which the dispatch takes
 * as unrouted; a group with fewer eligible experts than group_top is worth the
 * sum of those it has, and one with none does not stay.  A NaN or +infinity
 * among the logits makes a softmax's scores NaN, and so its keys where it is
 * keys that are compared; where logits are, renormalised weights come from the
 * chosen logits alone, and are NaN only where one of these is +infinity.
 *
 *   logits        [T,E] fp32 in; E <= EPDC_MAX_BINS
 *   bias          [E] fp32 in, or NULL
 *   num_groups    <= EPDC_MAX_GROUPS, divides E; topk_groups in [1, num_groups];
 *                 group_top 1 or 2
 *   scale         finite
 *   token_count   [1] int32 in, device memory, or NULL: tokens from
 *                 token_count[0] on (a batch's padding) are not read; their
 *                 ids are -1 and their weights 0
 *   topk_idx      [T,K] int64 out; topk_weights [T,K] fp32 out
 *                 (K <= EPDC_MAX_TOPK)
 */
int ep_route(const float* logits, int64_t num_tokens, int num_experts, int num_topk, int score,
             const float* bias, int num_groups, int topk_groups, int group_top, int renormalize,
             float scale, const int32_t* token_count, int64_t* topk_idx, float* topk_weights,
             hipStream_t stream);

/*
 * Gradient of ep_route's weights:
 *   dlogits[t,:] from dweights[t,:], the choice being constant.  With S the
 *   sum of the chosen s (1 without renormalize) and s_k, d_k slot k's,
 *   ds_k = scale / S * (d_k - [renormalize] sum_j d_j s_j / S)
 *   sigmoid: dlogits[e] = ds_k s_k (1 - s_k) for the chosen, else 0
 *   softmax: dlogits[e] = s[e] (ds[e] - sum_j ds_j s_j), ds = 0 unless chosen
 * In 64 bits, rounded once to fp32.  Slots whose id lies outside [0, E) are
 * skipped; a token without any has zeros, whatever its logits.  An expert that
 * two slots name gets the sum of both.  Where S is 0 dlogits is 0.
 *
 *   dweights  [T,K] fp32 in; logits [T,E] fp32 in; topk_idx [T,K] int64 in
 *   dlogits   [T,E] fp32 out
 */
int ep_route_backward(const float* dweights, const float* logits, const int64_t* topk_idx,
                      int64_t num_tokens, int num_experts, int num_topk, int score,
                      int renormalize, float scale, float* dlogits, hipStream_t stream);

/*
 * ep_dispatch_permute for rows that are in 8 bits already, as ep_rms_norm
 * makes them: codes and scale words move unchanged to every send row,
 *   send_q[token_row[t,k],:] = q[t,:],  send_scale[token_row[t,k],:] = scale[t,:].
 *
 *   q            [T,H] bytes in (16-byte aligned), H a multiple of 128
 *   scale        [T,scale_words] 32-bit words in; scale_words >= 0 (H/128 for
 *                one fp32 scale per 128 channels)
 *   token_row    [T,K] int32 in; entries outside [0, capacity) are skipped
 *   send_q       [capacity,H] bytes out (16-byte aligned)
 *   send_scale   [capacity,scale_words] out
 * Rows that no slot names are left as they are.
 */
int ep_dispatch_permute_quantized(const void* q, const void* scale, int scale_words,
                                  int64_t num_tokens, int hidden, const int32_t* token_row,
                                  int num_topk, int64_t num_send_capacity, void* send_q,
                                  void* send_scale, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EPDC_ROUTER_H */
