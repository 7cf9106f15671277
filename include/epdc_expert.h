/*
 * epdc_expert.h - the expert side of an MoE layer on one MI355X (gfx950).
 *
 * Second header of libepdc.so: what runs between the dispatch and the combine
 * of epdc.h.  The experts' products for a few rows (bf16 or 4-bit weights), a
 * whole expert layer for a few tokens in two or three launches, the gated
 * activation with an 8-bit checkpoint for its backward pass, and the gradient
 * of the combine.
 *
 * The conventions are those of epdc.h: device pointers to row-major,
 * contiguous arrays; the caller owns every buffer; the library allocates
 * nothing, keeps no state and never synchronizes; a call validates its
 * arguments on the host, returns a negative ep_status_t before anything is
 * enqueued if one is bad, and otherwise only enqueues kernels on `stream`.
 * The arrays belong to the current device.  A pointer to an empty array may
 * be NULL.  Outputs must not overlap inputs unless a call says so.
 */
#ifndef EPDC_EXPERT_H
#define EPDC_EXPERT_H

#include "epdc.h"

#ifdef __cplusplus
extern "C" {
#endif

#define EPDC_EXPERT_ABI_VERSION 1
/* Rows (or token slots T*K) the few-row products take, and tokens. */
#define EPDC_FEW_SLOTS 1024
#define EPDC_FEW_TOKENS 128
/* Channels (either side) of a few-row product, and bytes of one matrix. */
#define EPDC_FEW_CHANNELS 65536
#define EPDC_FEW_MATRIX_BYTES 0x7fffffff

/* Version of this header's ABI (EPDC_EXPERT_ABI_VERSION). */
int ep_expert_abi_version(void);

/*
 * Formats of a weight matrix [N, K] (N outputs, K input channels).  The 4-bit
 * formats hold channel 2j in the low half of byte j of a row and channel 2j+1
 * in the high half, and one scale for every `group` channels of a row:
 *   EP_W_BF16  [N, K] bf16; group 0, no scales;
 *   EP_W_INT4  [N, K/2] bytes; the code c stands for (c - 8) * scale, scales
 *              [N, K/group] bf16, group 32, 64 or 128;
 *   EP_W_FP4   [N, K/2] bytes; the code is an e2m1 float (sign, two exponent
 *              bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), times
 *              2^(byte - 127); scales [N, K/32] bytes (the byte 255 stands for
 *              NaN), group 32: the OCP microscaling format MXFP4.  Values of
 *              2^128 and more (bytes 253 and 254) read as infinities.
 * The channels K of a 4-bit matrix are a multiple of 128, of a bf16 one of 8.
 * E matrices of one shape lie one after the other.
 */
typedef enum {
    EP_W_BF16 = 0,
    EP_W_INT4 = 1,
    EP_W_FP4 = 2
} ep_weight_fmt_t;

/*
 * bf16 rows to 4-bit codes and scales.  With amax the largest magnitude of a
 * group:
 *   EP_W_INT4  scale = bf16(fp32(amax / 7)), code = 8 + rint(w / scale)
 *              (ties to even, the quotient in fp32, clamped to [-8, 7]);
 *   EP_W_FP4   scale = the smallest power of two >= fp32(amax / 6), at least
 *              2^-127; code = the nearest e2m1 value of w / scale, ties to the
 *              even code, sign kept.
 * A group of zeros (for int4 also one whose scale rounds to 0) gets the codes
 * of 0 and a zero scale (byte 0).  A group that holds a NaN or an infinity
 * gets the codes of 0 and a NaN scale, so that all of it reads as NaN.
 *
 *   w      [num_rows, channels] bf16 in (16-byte aligned)
 *   q      [num_rows, channels/2] bytes out (16-byte aligned)
 *   scale  [num_rows, channels/group] out (16-byte aligned)
 */
int ep_quantize_w4(const void* w, int64_t num_rows, int channels, int weight_fmt, int group,
                   void* q, void* scale, hipStream_t stream);

/*
 * Products of a few rows with their experts' matrices:
 *   y[r,:] = bf16( W[row_expert[r]] x[r,:] ),
 * products and sums in fp32, rounded once.  The weights of an expert that
 * several rows name are read once for 4 to 48 of them, by the sizes.  Rows whose
 * id lies outside [0, E) get +0.
 * An int4 product sums (c - 8) / 16 * x over a scale group in fp32 before the
 * scale: with every channel below 2^122 in magnitude no such sum leaves fp32,
 * whatever the codes and the group.  Larger finite channels may give infinities
 * or NaN.
 *
 *   x           [num_rows, channels] bf16 in (16-byte aligned)
 *   row_expert  [num_rows] int32 in, or NULL when num_experts == 1 (all 0)
 *   num_rows    <= EPDC_FEW_SLOTS
 *   w, w_scale  [E, out_channels, ...] in the format weight_fmt / group
 *               (16-byte aligned; w_scale NULL for bf16)
 *   y           [num_rows, out_channels] bf16 out (16-byte aligned)
 * out_channels is a multiple of 8; E <= EPDC_MAX_BINS; both channel counts
 * <= EPDC_FEW_CHANNELS and one matrix's bytes <= EPDC_FEW_MATRIX_BYTES.
 */
int ep_expert_matvec(const void* x, const int32_t* row_expert, int64_t num_rows, int num_experts,
                     int out_channels, int channels, int weight_fmt, int group, const void* w,
                     const void* w_scale, void* y, hipStream_t stream);

/*
 * Bytes of workspace ep_moe_tokens needs.  It holds the list of the experts in
 * use and the activations h; nothing in it has to be cleared, and nothing is
 * kept in it from one call to the next.  Calls that may overlap in time must
 * use different workspaces.  0 for sizes that the call rejects in every format
 * of the weights.
 */
size_t ep_moe_tokens_workspace_bytes(int64_t num_tokens, int num_topk, int hidden, int inner);

/*
 * A whole expert layer for a few tokens, in two launches, or three where the
 * sum over a token's experts is one of its own: with e = topk_idx[t,k] -
 * first_expert, for every slot whose e lies in [0, E_local),
 *   h[t,k,:] = silu(g) * u,  g = W13[e][0:I] x[t],  u = W13[e][I:2I] x[t]
 *   out[t,:] = bf16( sum_k w[t,k] * (W2[e] h[t,k,:]) + bias0[t,:] + bias1[t,:] )
 * silu(g) = g / (1 + exp(-g)).  Products and sums are in fp32: each slot's
 * output is multiplied by its weight in fp32 and added in ascending k from
 * +0.0, the biases that are given after it, bias0 first, as in ep_combine, but
 * without the rounding of a slot's output to bf16.  h is carried as the sum of
 * two bf16 numbers (off by at most 2^-17 of it).  Slots of other ids (-1, or
 * another GPU's experts) are skipped; a token with no local slot gives +0 plus
 * the biases.
 * The result does not depend on the order in which workgroups run.
 *
 *   x             [T,H] bf16 in (16-byte aligned)
 *   topk_idx      [T,K] int64 in; topk_weights [T,K] fp32 in
 *   num_tokens    T <= EPDC_FEW_TOKENS, and T*K <= EPDC_FEW_SLOTS
 *   w13, w13_scale  [E_local, 2I, H] in the format w13_fmt / w13_group: the I
 *                 gate rows, then the I up rows
 *   w2, w2_scale  [E_local, H, I] in the format w2_fmt / w2_group
 *   bias0, bias1  [T,H] bf16 in, or NULL (16-byte aligned)
 *   out           [T,H] bf16 out (16-byte aligned)
 *   workspace     ep_moe_tokens_workspace_bytes(T, K, H, I) bytes, 256-byte
 *                 aligned
 * H and I are multiples of 8 (of 128 where they are the channels of a 4-bit
 * matrix); the limits of ep_expert_matvec hold for both matrices, that on the
 * channels of an int4 product for x and for h.
 */
int ep_moe_tokens(const void* x, const int64_t* topk_idx, const float* topk_weights,
                  int64_t num_tokens, int num_topk, int hidden, int inner, int first_expert,
                  int num_local_experts, int w13_fmt, int w13_group, const void* w13,
                  const void* w13_scale, int w2_fmt, int w2_group, const void* w2,
                  const void* w2_scale, const void* bias0, const void* bias1, void* out,
                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Gated activation of the rows between an expert's two products, with a
 * checkpoint of its input in 8 bits for the backward pass:
 *   h[r,i] = bf16( silu(g) * u ),  g = gate_up[r,i],  u = gate_up[r,I+i]
 *   q, scale = e4m3 codes and one fp32 scale per 128 channels of gate_up[r,:]:
 *              amax = max |x|, scale = fp32(amax * fp32(1/448)), code =
 *              e4m3(fp32(x / scale)).
 * The rounding of the codes, zeros, NaN and infinities follow
 * ep_dispatch_permute's fp8 form, whose scale is fp32(amax / 448), at most one
 * unit in the last place from this one.  The product is what PyTorch computes
 * for amax / 448.0 on the GPU, so that q and scale equal a checkpoint made
 * there.  A user keeps q and scale (2I + I/16 bytes a row) instead of gate_up
 * and h (6I bytes).
 *
 *   gate_up    [num_rows, 2I] bf16 in (16-byte aligned)
 *   row_count  [1] int32 in, device memory, or NULL: rows from row_count[0] on
 *              are neither read nor written (expert_offsets + bins of
 *              ep_regroup_by_expert gives the rows in use of its buffers)
 *   h          [num_rows, I] bf16 out (16-byte aligned)
 *   q          [num_rows, 2I] e4m3 codes out (16-byte aligned)
 *   scale      [num_rows, 2I/128] fp32 out
 * I is a multiple of 128.
 */
int ep_swiglu_fp8(const void* gate_up, int64_t num_rows, int inner, const int32_t* row_count,
                  void* h, void* q, float* scale, hipStream_t stream);

/*
 * Backward pass of ep_swiglu_fp8 from its checkpoint: with g and u the values
 * code * scale that the checkpoint stands for and s = 1 / (1 + exp(-g)),
 *   d_gate_up[r,i]   = bf16( dh * u * s * (1 + g * (1 - s)) )
 *   d_gate_up[r,I+i] = bf16( dh * g * s )
 *   h[r,i]           = bf16( g * s * u )   (the second product's weight
 *                      gradient needs it; not written when h is NULL)
 *
 *   dh         [num_rows, I] bf16 in (16-byte aligned)
 *   q, scale   the checkpoint; row_count as above
 *   d_gate_up  [num_rows, 2I] bf16 out (16-byte aligned)
 */
int ep_swiglu_fp8_backward(const void* dh, const void* q, const float* scale, int64_t num_rows,
                           int inner, const int32_t* row_count, void* d_gate_up, void* h,
                           hipStream_t stream);

/*
 * Gradient of ep_combine.  For every row r that a slot of token t names,
 *   dy[r,:] = bf16( c * dout[t,:] ),  c = sum of w[t,k] over t's slots with
 *             token_row[t,k] == r (fp32, ascending k; c = 1 with no weights)
 *   dw[t,k] = <dout[t,:], y[token_row[t,k],:]> in fp32, 0 for slots with no
 *             row.
 * The sums run in a fixed order.  The gradient of a bias is dout itself.
 * Rows that no slot names (padding, spare capacity) are left as they are: a
 * caller who reads those clears them, and again for every new token_row, since
 * a row that a slot named before may be one that none names now.  The slots of
 * two tokens must not name the same row (no layout of epdc.h does).  The
 * gradient of the dispatch is ep_combine with topk_weights == NULL.  The way
 * back from the expert-major rows of ep_regroup_by_expert is ep_combine over its
 * row_map, so that its gradient is this call with token_row = row_map, and the
 * regroup's is ep_combine over row_map with topk_weights == NULL.
 *
 *   dout          [T,H] bf16 in (16-byte aligned)
 *   y             [num_rows,H] bf16 in (16-byte aligned); may be NULL when dw
 *                 is
 *   token_row     [T,K] int32 in; rows outside [0, num_rows) are skipped
 *   topk_weights  [T,K] fp32 in, or NULL (the unweighted combine; dw must then
 *                 be NULL)
 *   dy            [num_rows,H] bf16 out (16-byte aligned)
 *   dw            [T,K] fp32 out, or NULL
 */
int ep_combine_backward(const void* dout, const void* y, int64_t num_rows,
                        const int32_t* token_row, const float* topk_weights, int64_t num_tokens,
                        int num_topk, int hidden, void* dy, float* dw, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EPDC_EXPERT_H */
