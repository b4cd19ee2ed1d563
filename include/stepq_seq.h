/*
 * stepq_seq.h -- C ABI of libstepq.so around the packed decode step: how a
 * request's state comes into being and how its beams are kept.
 *
 *   stepq_linear_prefill   linear attention with one decay per head over ragged
 *                          prompts (chunked form); leaves the final states that
 *                          stepq_pack admits into the packed pool
 *   stepq_linear_step      the same recurrence for one token of every request,
 *                          on binary32 states
 *   stepq_beam_select      beam search's selection over beams and vocabulary
 *   stepq_beam_reorder     the matching reordering of state slots, packed or not
 *
 * Conventions are those of stepq.h: the caller owns every device buffer, calls
 * enqueue on the caller's stream and return without synchronising, allocating
 * or copying between host and device (they may be captured into a graph),
 * argument checks run before any launch and have no side effects, no exception
 * crosses the ABI, and work runs on the HIP device that is current, on which every
 * buffer has to lie (not checked here; the Python bindings do).  q, k, v, o,
 * states, regions and workspaces are 16-byte aligned, logits and arrays of 32-bit
 * values (lengths, ids, beta, gate, scores) as their elements.  Two calls that use
 * one workspace must be ordered; its contents need no initialisation and mean
 * nothing afterwards.
 *
 * What does not join: stepq_decode_step is the delta rule on dense binary32 q, k
 * and v of every value head.  After prompts of 16-bit inputs or shared key heads the
 * caller widens them and repeats key heads for it at every token
 * (stepq_linear_step takes them as they are, on binary32 states), and the states of
 * the additive rule can be packed and unpacked, but only the calls here continue
 * them.
 */
#ifndef STEPQ_SEQ_H
#define STEPQ_SEQ_H

#include "stepq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of q, k, v, o (linear attention) and of the logits (beams). */
typedef enum {
  STEPQ_F32 = 0,
  STEPQ_BF16 = 1,
  STEPQ_F16 = 2
} stepq_dtype;

/* State update of one token, M a D x D matrix with row i = key channel and
 * column j = value channel, a the retention, b = beta:
 *   additive:  M_t = a_t M_{t-1} + k_t v_t^T
 *   delta:     M_t = a_t M_{t-1} + b_t k_t (v_t - a_t M_{t-1}^T k_t)^T
 * and o_t = M_t^T q_t for both.  The delta rule is the one of
 * stepq_decode_step under the per-head gate. */
typedef enum {
  STEPQ_RULE_ADDITIVE = 0,
  STEPQ_RULE_DELTA = 1
} stepq_rule;

typedef struct {
  int32_t num_heads;     /* H >= 1 value heads; every value head has a state */
  int32_t num_qk_heads;  /* Hk >= 1, divides H: value head h reads q and k of head h / (H / Hk) */
  int32_t d;             /* key = value channels per head: 16, 32, 64 or 128 */
  int32_t rule;          /* stepq_rule */
  int32_t dtype;         /* stepq_dtype of q, k, v and o */
} stepq_linear_desc;

/* Bytes that are enough as stepq_linear_prefill's workspace for every call of up to
 * `batch` requests of up to `total_tokens` tokens together; 0 where no such call
 * needs one, for an invalid desc or a negative size. */
size_t stepq_linear_workspace_bytes(const stepq_linear_desc *desc, int32_t batch, int64_t total_tokens);

/* Bytes stepq_linear_prefill asks for in a call of exactly these sizes; 0 for a call
 * that runs in one launch, as those of 16-bit inputs at d = 64 and 128 with many
 * (request, head) pairs do (the workspace may then be NULL). */
size_t stepq_linear_prefill_bytes(const stepq_linear_desc *desc, int32_t batch, int64_t total_tokens);

/* Prompts.  Request b's tokens are rows cu_seqlens[b] .. cu_seqlens[b+1]-1 of
 * q, k, v, o, beta and gate (device int32 [batch+1], non-decreasing, within
 * [0, total_tokens]; entries outside are clamped).  Any length is allowed,
 * 0 and 1 among them: an empty request leaves the state it starts from.
 *   q, k: [total_tokens][Hk][D], v, o: [total_tokens][H][D] of desc->dtype;
 *         *_stride is the distance of two tokens in elements (>= heads * D, at most
 *         2^24, a multiple of 16 bytes), so slices of one fused projection need no copy.
 *         q and k are used as given.  o must not overlap an input.
 *   beta: float [total_tokens][H], NULL for the additive rule.
 *   gate: float [total_tokens][H], linear retention a in [0, 1]; 0 clears the
 *         state.
 *   slot_ids: device int32 [batch], distinct; request b's state is slot
 *         slot_ids[b] of state, float [num_slots][H][D][D].  A request whose id
 *         lies outside [0, num_slots) has its rows of o written as NaN and
 *         touches no state.
 *   resume: device uint8 [batch]: non-zero continues from the slot's state,
 *         zero starts from a zero state.  NULL: every request starts from zero.
 * The slots receive the states after the last token; a pool whose slots are
 * these states is also the packed pool of a layout whose heads are all 32 bits
 * wide, and stepq_pack takes them when slot_ids is 0 .. batch-1.
 * States, sums, retentions and the operands of products are held in binary32 (of
 * 16-bit inputs as three bfloat16 parts); o is rounded once.  A value
 * that is not finite spoils what depends on it and may spoil o of the tokens
 * before it in its chunk of 64, but no other request. */
stepq_status stepq_linear_prefill(const stepq_linear_desc *desc, int32_t batch, int64_t total_tokens,
                                  const int32_t *cu_seqlens, const void *q, int64_t q_stride, const void *k,
                                  int64_t k_stride, const void *v, int64_t v_stride, const float *beta,
                                  const float *gate, const int32_t *slot_ids, int32_t num_slots,
                                  const uint8_t *resume, float *state, void *o, int64_t o_stride,
                                  void *workspace, size_t workspace_bytes, void *stream);

/* One token of every request: row b of q, k, v, o, beta and gate (otherwise as
 * above) updates slot slot_ids[b] in place.  A request whose id lies outside
 * [0, num_slots) has its row of o written as NaN. */
stepq_status stepq_linear_step(const stepq_linear_desc *desc, int32_t batch, const int32_t *slot_ids,
                               int32_t num_slots, const void *q, int64_t q_stride, const void *k,
                               int64_t k_stride, const void *v, int64_t v_stride, const float *beta,
                               const float *gate, float *state, void *o, int64_t o_stride, void *stream);

/* Bytes stepq_beam_select needs as workspace; 0 for sizes it refuses. */
size_t stepq_beam_workspace_bytes(int32_t batch, int32_t beams, int32_t vocab, int32_t num_out);

/* Selection.  Beam i of request b is row r = b * beams + i of logits (dtype,
 * logits_stride >= vocab elements from row to row), of scores (float, the beam's sum of log probabilities) and of
 * finished.  Token t continues it at score scores[r] + (x_t - max x) - log sum
 * exp(x - max x); a beam with finished[r] != 0 has one continuation, eos_token,
 * at scores[r].  The num_out best of a request, 1 .. 64, are written in order:
 *   tokens, parents: int32 [batch][num_out] (parents: the beam, 0 .. beams-1)
 *   out_scores: float [batch][num_out]
 * The order is by score; equal scores go to the lower beam, then to the larger
 * logit, then to the lower token.  A logit of -inf or NaN bans its token, and a
 * row whose logits are all banned, or whose score is -inf or NaN, has no
 * continuation; among logits of +inf the probability is shared.  Where a
 * request has fewer than num_out continuations the rest is token -1, parent -1,
 * score -inf.  beams: 1 .. 64.  finished may be NULL. */
stepq_status stepq_beam_select(int32_t batch, int32_t beams, int32_t vocab, int32_t num_out,
                               const void *logits, int32_t dtype, int64_t logits_stride, const float *scores,
                               const uint8_t *finished, int32_t eos_token, int32_t *tokens, int32_t *parents,
                               float *out_scores, void *workspace, size_t workspace_bytes, void *stream);

/* A buffer of slots, for instance a packed pool, its scale table, or the pool
 * of another layer: slot s is the bytes [s * slot_bytes, (s + 1) * slot_bytes)
 * from base (device, 16-byte aligned; slot_bytes a positive multiple of 16). */
typedef struct {
  void *base;
  size_t slot_bytes;
} stepq_region;

#define STEPQ_MAX_REGIONS 128

/* Reordering.  parents: device int32 [batch][beams], the beam that each new
 * beam continues (0 .. beams-1), or anything else for a new beam that continues
 * none.  A parent's first child keeps the parent's slot, so a beam that goes on
 * alone is not moved; every further child, in ascending order, takes the slot of
 * the next beam without children (ascending), into which the parent's slot is
 * copied in every region; a new beam without a parent takes such a slot without
 * a copy.  slot_ids: device int32 [batch][beams], distinct over the whole call.
 * new_slot_ids: device int32 [batch][beams], written, a permutation of each
 * request's slot_ids; it must not overlap slot_ids or parents.  Ids outside
 * [0, num_slots) are permuted like the others and nothing is copied from or to
 * them.  regions is a host array, read during the call.  beams: 1 .. 64. */
stepq_status stepq_beam_reorder(int32_t batch, int32_t beams, const int32_t *slot_ids, const int32_t *parents,
                                int32_t num_slots, const stepq_region *regions, int32_t num_regions,
                                int32_t *new_slot_ids, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* STEPQ_SEQ_H */
