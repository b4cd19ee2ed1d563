// Internal declarations shared by the host API (linear_api.cpp) and the
// gfx950 kernels (linear_kernels.hip) of the linear-attention entry points.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/stepq_seq.h"

namespace stepq {

constexpr int kChunk = 64;   // tokens of one chunk of the chunked form

struct LinearArgs {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride;            // elements from token to token
  int64_t k_stride;
  int64_t v_stride;
  const float* beta;           // nullptr: additive rule
  const float* gate;
  const int32_t* slot_ids;
  const int32_t* cu_seqlens;   // prefill only
  const uint8_t* resume;       // prefill only; nullptr: all from zero
  float* state;
  void* o;
  int64_t o_stride;
  int64_t total_tokens;        // prefill only
  int32_t batch;
  int32_t num_slots;
  int32_t H;
  int32_t rep;                 // value heads per key head
  uint8_t* workspace;
  int32_t segment;             // prefill: chunks of a segment, 0: none (see segment_chunks)
  bool apart;                  // prefill of 16-bit inputs: see chunks_apart
};

// Chunks of all requests together: request b's chunks start at index
// cu_seqlens[b] / 64 + b, so that no table of them is needed.  From b to b + 1 the
// index grows by at least the ceil((cu[b + 1] - cu[b]) / 64) chunks of request b.
inline int64_t max_chunks(int64_t total_tokens, int32_t batch) { return total_tokens / kChunk + batch; }

// How a prefill of 16-bit inputs is spread over the chip, by (request, head) pairs.  us of
// calls with both sides built, requests of one length, 16 heads or one request:
//
//   all in one launch, a workgroup for every pair, against chunk matrices from a launch
//   of their own and several workgroups a pair (the walk of D = 128 under the delta rule):
//     pairs                          64          96         128         144         160
//     bfloat16, 1000 tokens       162 : 141   162 : 124   163 : 130               164 : 166
//     bfloat16, 4000 tokens                               624 : 533   627 : 636   626 : 653
//     binary16, 1000 tokens       204 : 162   205 : 159   205 : 172               205 : 297
//     binary16, 4000 tokens                               787 : 691   788 : 1164  785 : 1198
//   D = 64 under the delta rule: one launch is ahead at every number of pairs (1 pair of
//   4096 tokens 343 : 352, 128 of 1024 92 : 122; binary16 428 : 458, 114 : 153), and so it is
//   under the additive rule where there are no segments (1 pair of 511 tokens, D = 128,
//   41 : 44; 120 pairs 44 : 56; D = 64, 28 : 32 and 29 : 41).
//   Below D = 64 a pair is too little for a workgroup of four waves: always apart.
//
//   all in one launch against segments (additive rule):
//     D = 128, bfloat16: 128 pairs of 4000 tokens 304 : 296, 144 pairs 305 : 344, 160 307 : 363;
//     D = 64: 128 pairs 207 : 112, 176 pairs 225 : 162, 256 pairs of 1024 57 : 72.
constexpr int64_t kMostApart = 128;
constexpr int64_t most_segmented(int d) { return d == 128 ? 128 : 255; }

constexpr bool ever_apart(int d, bool delta) { return d < 64 || (d == 128 && delta); }

// Whether a prefill's chunk matrices come from a launch of their own.  Prompts of a chunk
// or less go in one launch: 37 tokens of 48 heads 14.4 us a call against 17.7 in two.
inline bool chunks_apart(const stepq_linear_desc& d, int64_t total_tokens, int32_t batch) {
  if (d.dtype == STEPQ_F32 || d.d < 64) return true;
  return ever_apart(d.d, d.rule == STEPQ_RULE_DELTA) && static_cast<int64_t>(batch) * d.num_heads <= kMostApart &&
         total_tokens > static_cast<int64_t>(batch) * kChunk;
}

constexpr int kLds = 163840;         // bytes of a compute unit's LDS
constexpr int kTri = 6 * 1024;       // bytes of a lower triangle's operands in one part
constexpr int kParts = 3;            // bfloat16 parts of a binary32 value

// A (chunk, head) of the workspace of 16-bit inputs: G, G_C / G, A, the system for U.
constexpr int block_bytes(bool delta) { return 2 * kChunk * 4 + (delta ? 2 : 1) * kParts * kTri; }

// LDS of a walk apart from its chunk matrices, 16 `waves` columns of a head: K and Q in
// `parts` parts, V, the chunk matrices.
constexpr int apart_lds(int d, int parts, bool delta, int waves) {
  const int row = 2 * (d < 32 ? 32 : d), vrow = 32 * waves < 64 ? 64 : 32 * waves;
  return kChunk * (2 * parts * row + vrow) + block_bytes(delta);
}

// Waves (columns / 16) of such a workgroup: as few as the chip holds workgroups for at once.
constexpr int apart_waves(int d, int parts, bool delta, int64_t pairs) {
  for (int waves = 1; waves < 4 && 16 * waves < d; waves *= 2)
    if (pairs * (d / (16 * waves)) <= static_cast<int64_t>(256) * (kLds / apart_lds(d, parts, delta, waves))) return waves;
  return d < 64 ? d / 16 : 4;
}

// Segments a long prompt of few heads is walked in (additive rule, 16-bit inputs, D >=
// 64, an average of 512 tokens or more): at least 4 chunks each, and so long that the
// heads' segments are some 768 workgroups.  The same index rule as for chunks.
// 512 and 1024 workgroups instead, us against those of 768: 16384 tokens of 32 heads of 128
// 300 and 321 : 314, of 16 heads 146 and 166 : 164, 32768 of 48 heads 913 and 761 : 773 (11
// segments of 48 heads are 528, more than the 512 that the chip holds at once),
// 16384 of 32 heads of 64 125 and 137 : 116, binary16 410 and 440 : 441.
inline int32_t segment_chunks(const stepq_linear_desc& d, int64_t total_tokens, int32_t batch) {
  if (d.rule != STEPQ_RULE_ADDITIVE || d.dtype == STEPQ_F32 || d.d < 64) return 0;
  if (static_cast<int64_t>(batch) * d.num_heads > most_segmented(d.d) || total_tokens < static_cast<int64_t>(batch) * 512) return 0;
  const int64_t wanted = (768 + d.num_heads - 1) / d.num_heads, chunks = total_tokens / kChunk;
  const int64_t n = (chunks + wanted - 1) / wanted;
  return static_cast<int32_t>(n < 4 ? 4 : n);
}
inline int64_t max_segments(int64_t total_tokens, int32_t batch, int32_t segment) {
  return total_tokens / (static_cast<int64_t>(segment) * kChunk) + batch;
}
constexpr int kSegmentHead = 16;   // floats after a segment's state: its retention, and padding

// Workspace bytes of one (chunk, value head).
inline size_t chunk_bytes(int rule, int dtype) {
  const bool delta = rule == STEPQ_RULE_DELTA;
  if (dtype == STEPQ_F32) return sizeof(float) * ((delta ? 2 : 1) * kChunk * kChunk + 2 * kChunk);
  return block_bytes(delta);
}

inline size_t chunks_workspace(const stepq_linear_desc& d, int64_t total_tokens, int64_t batch) {
  return static_cast<size_t>(total_tokens / kChunk + batch) * d.num_heads * chunk_bytes(d.rule, d.dtype);
}
inline size_t segments_workspace(const stepq_linear_desc& d, int64_t segments) {
  return static_cast<size_t>(segments) * d.num_heads * (static_cast<size_t>(d.d) * d.d + kSegmentHead) * sizeof(float);
}

// Workspace bytes of a call of these sizes.
inline size_t call_workspace(const stepq_linear_desc& d, int64_t total_tokens, int32_t batch) {
  const int32_t segment = segment_chunks(d, total_tokens, batch);
  if (segment > 0) return segments_workspace(d, max_segments(total_tokens, batch, segment));
  return chunks_apart(d, total_tokens, batch) ? chunks_workspace(d, total_tokens, batch) : 0;
}

// Workspace bytes that are enough for any call of up to these sizes: of those that use
// one, the one of the most requests.
inline size_t most_workspace(const stepq_linear_desc& d, int64_t total_tokens, int32_t batch) {
  const bool delta = d.rule == STEPQ_RULE_DELTA;
  const auto fewer = [&](int64_t pairs) { return batch < pairs / d.num_heads ? batch : pairs / d.num_heads; };
  if (d.dtype == STEPQ_F32 || d.d < 64) return chunks_workspace(d, total_tokens, batch);
  if (delta) return ever_apart(d.d, delta) && fewer(kMostApart) > 0 ? chunks_workspace(d, total_tokens, fewer(kMostApart)) : 0;
  const int64_t few = fewer(most_segmented(d.d)), wanted = (768 + d.num_heads - 1) / d.num_heads;
  const int64_t all = total_tokens / (4 * kChunk);
  return few > 0 ? segments_workspace(d, (all < wanted ? all : wanted) + few) : 0;
}

hipError_t launch_linear_prefill(const stepq_linear_desc& d, const LinearArgs& a, hipStream_t s);
hipError_t launch_linear_step(const stepq_linear_desc& d, const LinearArgs& a, hipStream_t s);

}  // namespace stepq
