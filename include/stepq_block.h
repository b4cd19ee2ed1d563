/*
 * stepq_block.h -- C ABI of libstepq.so for the block around a recurrent state, in
 * training and in serving with drafted tokens:
 *
 *   stepq_scan_forward     a gated linear recurrence, channel by channel, over ragged
 *                          prompts
 *   stepq_scan_backward    its gradients
 *   stepq_scan_step        one token of every request
 *   stepq_norm_forward     the norms before and after a block, with its gate, its residual
 *                          scale and the residual sum
 *   stepq_norm_backward    their gradients
 *   stepq_verify_drafts    which drafted tokens a target model accepts, and the token after
 *                          them, from given random numbers
 *
 * Conventions are those of stepq_seq.h: the caller owns every device buffer, calls
 * enqueue on the caller's stream and return without synchronising, allocating or copying
 * between host and device (they may be captured into a graph), argument checks run before
 * any launch and have no side effects, no exception crosses the ABI, and work runs on the
 * HIP device that is current, on which every buffer has to lie (not checked here; the
 * Python bindings do).  Buffers are aligned as their elements, workspaces and what a
 * forward pass saves to 16 bytes.  A *_stride is the distance of two tokens in elements,
 * at least a token's width, so slices of one fused projection need no copy, and at most 2^24
 * (stepq_scan_*, whose kernels reach a piece's rows by offsets of 32 bits), 2^40 (stepq_norm_*) or 2^38
 * (stepq_verify_drafts); others are STEPQ_ERR_INVALID_ARG.  Outputs must not overlap inputs or
 * each other unless said otherwise.  Two calls that use one workspace
 * must be ordered; its contents need no initialisation and mean nothing afterwards.
 */
#ifndef STEPQ_BLOCK_H
#define STEPQ_BLOCK_H

#include "stepq_seq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The gated linear recurrence.  With s the logistic function, for every channel
 *   a_t = exp(-rate s(gate_a_t) softplus(decay))        the retention
 *   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) s(gate_x_t) x_t
 *   y_t = h_t
 * States, retentions and sums are held in binary32; y is rounded once. */
typedef struct {
  int32_t width;    /* channels, 1 .. 2^20 */
  int32_t dtype;    /* stepq_dtype of x, the gates, y and their gradients */
  float rate;       /* finite, > 0 */
} stepq_scan_desc;

/* Bytes that are enough as workspace of stepq_scan_forward and stepq_scan_backward for every
 * call of up to `batch` requests of up to `total_tokens` tokens together; 0 where no such
 * call needs one, for an invalid desc or a negative size. */
size_t stepq_scan_workspace_bytes(const stepq_scan_desc *desc, int32_t batch, int64_t total_tokens);

/* Bytes a forward pass of exactly these sizes saves for its backward pass (0 as above). */
size_t stepq_scan_saved_bytes(const stepq_scan_desc *desc, int32_t batch, int64_t total_tokens);

/* Prompts.  Request b's tokens are rows cu_seqlens[b] .. cu_seqlens[b+1]-1 (device int32
 * [batch+1], non-decreasing, within [0, total_tokens]; entries outside are clamped).  Any
 * length is allowed, 0 and 1 among them: an empty request leaves the state it starts from.
 * Rows of no request are not touched.
 *   x, gate_a, gate_x, y: [total_tokens][width] of desc->dtype
 *   decay: float [width]
 *   slot_ids: device int32 [batch], distinct; request b's state is slot slot_ids[b] of
 *         state, float [num_slots][width].  A request whose id lies outside
 *         [0, num_slots) has its rows of y written as NaN and touches no state.
 *         slot_ids and state may both be NULL: every request starts from zero and its
 *         last state is not kept.
 *   resume: device uint8 [batch]: non-zero continues from the slot's state, zero
 *         starts from a zero state.  NULL: every request starts from zero.
 *   saved: what stepq_scan_backward reads, stepq_scan_saved_bytes; NULL where there
 *         is no backward pass.
 * A value that is not finite spoils what depends on it, and no other request or channel. */
stepq_status stepq_scan_forward(const stepq_scan_desc *desc, int32_t batch, int64_t total_tokens,
                                const int32_t *cu_seqlens, const void *x, int64_t x_stride, const void *gate_a,
                                int64_t gate_a_stride, const void *gate_x, int64_t gate_x_stride,
                                const float *decay, const int32_t *slot_ids, int32_t num_slots,
                                const uint8_t *resume, float *state, void *y, int64_t y_stride, void *saved,
                                size_t saved_bytes, void *workspace, size_t workspace_bytes, void *stream);

/* Gradients, from those of y and, where there are slots, of the states that requests end
 * with.  cu_seqlens, x, gate_a, gate_x, decay, slot_ids and resume are those of the forward
 * pass and saved is what it left.
 *   dy: [total_tokens][width] of desc->dtype
 *   dx, dgate_a, dgate_x: the same, written
 *   ddecay: float [width], written (not added to)
 *   dstate: float [num_slots][width]: request b's slot holds the gradient of the state that
 *         it ends with and receives that of the state that it starts from (0 where it
 *         starts from zero).  slot_ids and dstate may both be NULL: no state is kept.
 * A request whose id lies outside [0, num_slots) has its rows of dx, dgate_a and dgate_x
 * written as NaN and adds nothing to ddecay.  The same inputs give the same bits. */
stepq_status stepq_scan_backward(const stepq_scan_desc *desc, int32_t batch, int64_t total_tokens,
                                 const int32_t *cu_seqlens, const void *x, int64_t x_stride, const void *gate_a,
                                 int64_t gate_a_stride, const void *gate_x, int64_t gate_x_stride,
                                 const float *decay, const void *saved, size_t saved_bytes, const void *dy,
                                 int64_t dy_stride, const int32_t *slot_ids, int32_t num_slots,
                                 const uint8_t *resume, float *dstate, void *dx, int64_t dx_stride, void *dgate_a,
                                 int64_t dgate_a_stride, void *dgate_x, int64_t dgate_x_stride, float *ddecay,
                                 void *workspace, size_t workspace_bytes, void *stream);

/* One token of every request: row b of x, gate_a, gate_x and y (otherwise as above) updates
 * slot slot_ids[b] in place.  A request whose id lies outside [0, num_slots) has its row of
 * y written as NaN. */
stepq_status stepq_scan_step(const stepq_scan_desc *desc, int32_t batch, const int32_t *slot_ids, int32_t num_slots,
                             const void *x, int64_t x_stride, const void *gate_a, int64_t gate_a_stride,
                             const void *gate_x, int64_t gate_x_stride, const float *decay, float *state, void *y,
                             int64_t y_stride, void *stream);

/* The norms around a block.  For every token and head, a row of `width` values o of the block's
 * result, z of the gate and x of the residual stream:
 *   n = o rsqrt(mean o^2 + eps) post_weight     (post = 0: n = o)
 *   t = x + scale n act(z)                      written to out
 *   y = t rsqrt(mean t^2 + eps) pre_weight      written to normed (pre = 0: there is none)
 * act is z s(z) or s(z), s the logistic function; what is not given is left out: no gate, act
 * is 1, no residual, x is 0, no scale or weight, it is 1.  So post alone with a gate is the
 * gated norm behind a recurrent readout, pre alone with a residual is a residual sum and
 * the next block's norm.  Everything is worked out in binary32 (y from t before it is rounded)
 * and rounded once. */
typedef enum {
  STEPQ_GATE_SILU = 0,
  STEPQ_GATE_SIGMOID = 1
} stepq_gate_activation;

typedef struct {
  int32_t width;        /* values of a row, 1 .. 16384 */
  int32_t heads;        /* rows of a token, side by side, >= 1 */
  int32_t dtype;        /* stepq_dtype of all tensors of tokens */
  int32_t activation;   /* stepq_gate_activation */
  int32_t post;         /* 0 or 1 */
  int32_t pre;          /* 0 or 1 */
  float eps;            /* a normal number > 0 */
} stepq_norm_desc;

/* Tensors of tokens are [tokens][heads * width], tokens *_stride elements apart; weights and
 * scale are float [width], shared by the heads.  gate, residual, post_weight, scale and
 * pre_weight may be NULL; out may be NULL where pre is 1.  out and normed may each be the
 * buffer of block, gate or residual, at the same stride (not of each other).
 * tokens * heads is below 2^31.  A value that is not finite spoils its row alone; a row whose sum of
 * squares is beyond binary32's range is normalised to 0. */
stepq_status stepq_norm_forward(const stepq_norm_desc *desc, int64_t tokens, const void *block, int64_t block_stride,
                                const void *gate, int64_t gate_stride, const void *residual,
                                int64_t residual_stride, const float *post_weight, const float *scale,
                                const float *pre_weight, void *out, int64_t out_stride, void *normed,
                                int64_t normed_stride, void *stream);

/* Bytes stepq_norm_backward needs as workspace for up to `tokens` tokens; 0 for an invalid desc
 * or sizes it refuses. */
size_t stepq_norm_workspace_bytes(const stepq_norm_desc *desc, int64_t tokens);

/* Gradients.  block, gate, post_weight, scale and pre_weight are those of the forward pass; out
 * is what it wrote (pre = 0: not read, may be NULL).  d_out and d_normed are the gradients of
 * out and normed: d_normed is given exactly where pre is 1, and there d_out may be NULL.
 * Written: d_block; d_gate, where there is a gate; d_residual (NULL where it is not wanted);
 * and, float [width] each and NULL where not wanted, d_post_weight, d_scale and d_pre_weight
 * of weights that are given.  d_block, d_gate and d_residual may each be the buffer of
 * block, gate, out, d_out or d_normed, at the same stride (not of each other).  The same
 * inputs give the same bits. */
stepq_status stepq_norm_backward(const stepq_norm_desc *desc, int64_t tokens, const void *block, int64_t block_stride,
                                 const void *gate, int64_t gate_stride, const void *out, int64_t out_stride,
                                 const float *post_weight, const float *scale, const float *pre_weight,
                                 const void *d_out, int64_t d_out_stride, const void *d_normed,
                                 int64_t d_normed_stride, void *d_block, int64_t d_block_stride, void *d_gate,
                                 int64_t d_gate_stride, void *d_residual, int64_t d_residual_stride,
                                 float *d_post_weight, float *d_scale, float *d_pre_weight, void *workspace,
                                 size_t workspace_bytes, void *stream);

/* Bytes stepq_verify_drafts needs as workspace; 0 for sizes it refuses. */
size_t stepq_verify_workspace_bytes(int32_t batch, int32_t drafts, int32_t vocab);

/* Verification of drafted tokens.  Request b has num_drafts[b] of them (NULL: all `drafts`; clamped to
 * 0 .. drafts), draft_tokens[b][0 ..]; row b * (drafts + 1) + k of logits is the target's for the
 * token at place k (one more than there are drafts), row b * drafts + k of draft_logits the draft's.
 * With p and q the softmax of the two rows over temperature[b] (NULL: 1), drafted token d at
 * place k is accepted where all before it are and
 *     uniforms[b][k] q(d) < p(d)
 * Behind n accepted ones the next token is drawn from max(p - q, 0) where a draft was rejected at
 * place n (from p should nothing be left of it), from p where all were accepted: it is the first
 * one up to which the sum exceeds uniforms[b][drafts] times the whole.  So the tokens are distributed as
 * the target's own, whatever the draft; drafts = 0 draws a token.
 *   draft_logits NULL: the draft was certain of its tokens, q(d) = 1.
 *   temperature 0 (or less, or NaN): greedy.  p is the lowest of the tokens with the largest
 *     logit, a draft is accepted if it is that token, and draft_logits are not read.
 *   A logit of -inf or NaN bans its token; among logits of +inf the probability is shared.
 *     Where all of the target's row is banned nothing is accepted and the next token is -1.
 *   A drafted token outside of the vocabulary ends the request's drafts before it.
 * Written: accepted int32 [batch], n; tokens int32 [batch][drafts + 1], the accepted drafts, the
 * next token, and -1 behind it.  logits and draft_logits are of type dtype, their rows *_stride >=
 * vocab elements apart; draft_tokens int32 [batch][drafts]; uniforms float [batch][drafts + 1] in
 * [0, 1); temperature float [batch].  Probabilities are worked out and summed in binary64.
 * drafts: 0 .. 63. */
stepq_status stepq_verify_drafts(int32_t batch, int32_t drafts, int32_t vocab, const void *logits, int32_t dtype,
                                 int64_t logits_stride, const void *draft_logits, int64_t draft_logits_stride,
                                 const int32_t *draft_tokens, const int32_t *num_drafts, const float *temperature,
                                 const float *uniforms, int32_t *accepted, int32_t *tokens, void *workspace,
                                 size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* STEPQ_BLOCK_H */
