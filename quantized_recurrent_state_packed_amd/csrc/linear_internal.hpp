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
};

// Chunks of all requests together: request b's chunks start at index
// cu_seqlens[b] / 64 + b, so that no table of them is needed.  From b to b + 1 the
// index grows by at least the ceil((cu[b + 1] - cu[b]) / 64) chunks of request b.
inline int64_t max_chunks(int64_t total_tokens, int32_t batch) { return total_tokens / kChunk + batch; }

// (request, head) pairs from which one workgroup for each fills the chip.
constexpr int kFullChip = 256;

// Segments a long prompt of few heads is walked in (additive rule, 16-bit inputs, D >=
// 64, an average of 512 tokens or more): at least 4 chunks each, and so long that the
// heads' segments are some 768 workgroups.  The same index rule as for chunks.
inline int32_t segment_chunks(const stepq_linear_desc& d, int64_t total_tokens, int32_t batch) {
  if (d.rule != STEPQ_RULE_ADDITIVE || d.dtype == STEPQ_F32 || d.d < 64) return 0;
  if (static_cast<int64_t>(batch) * d.num_heads >= kFullChip || total_tokens < static_cast<int64_t>(batch) * 512) return 0;
  const int64_t wanted = (768 + d.num_heads - 1) / d.num_heads, chunks = total_tokens / kChunk;
  const int64_t n = (chunks + wanted - 1) / wanted;
  return static_cast<int32_t>(n < 4 ? 4 : n);
}
inline int64_t max_segments(int64_t total_tokens, int32_t batch, int32_t segment) {
  return total_tokens / (static_cast<int64_t>(segment) * kChunk) + batch;
}
constexpr int kSegmentHead = 16;   // floats after a segment's state: its retention, and padding

// Workspace bytes for segments of any call of up to these sizes.
inline size_t segment_workspace_bytes(const stepq_linear_desc& d, int64_t total_tokens, int32_t batch) {
  if (d.rule != STEPQ_RULE_ADDITIVE || d.dtype == STEPQ_F32 || d.d < 64) return 0;
  const int64_t wanted = (768 + d.num_heads - 1) / d.num_heads, all = total_tokens / (4 * kChunk);
  const int64_t few = kFullChip / d.num_heads + 1;
  const int64_t segments = (all < wanted ? all : wanted) + (batch < few ? batch : few);
  return static_cast<size_t>(segments) * d.num_heads * (static_cast<size_t>(d.d) * d.d + kSegmentHead) * sizeof(float);
}

// Workspace bytes of one (chunk, value head).
size_t chunk_bytes(int rule, int dtype);

hipError_t launch_linear_prefill(const stepq_linear_desc& d, const LinearArgs& a, hipStream_t s);
hipError_t launch_linear_step(const stepq_linear_desc& d, const LinearArgs& a, hipStream_t s);

}  // namespace stepq
