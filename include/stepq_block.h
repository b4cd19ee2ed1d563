/*
 * stepq_block.h -- C ABI of libstepq.so for the block around a recurrent state, in
 * training and in serving with drafted tokens:
 *
 *   stepq_scan_forward     a gated linear recurrence, channel by channel, over ragged
 *                          prompts
 *   stepq_scan_backward    its gradients
 *   stepq_scan_step        one token of every request
 *
 * Conventions are those of stepq_seq.h: the caller owns every device buffer, calls
 * enqueue on the caller's stream and return without synchronising, allocating or copying
 * between host and device (they may be captured into a graph), argument checks run before
 * any launch and have no side effects, no exception crosses the ABI, and work runs on the
 * HIP device that is current, on which every buffer has to lie (not checked here; the
 * Python bindings do).  Buffers are aligned as their elements, workspaces and what a
 * forward pass saves to 16 bytes.  A *_stride is the distance of two tokens in elements,
 * at least a token's width, so slices of one fused projection need no copy; outputs must
 * not overlap inputs or each other unless said otherwise.  Two calls that use one workspace
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

#ifdef __cplusplus
}
#endif

#endif /* STEPQ_BLOCK_H */
