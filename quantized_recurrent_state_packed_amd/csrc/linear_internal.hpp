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
};

// Chunks of all requests together: request b's chunks start at index
// cu_seqlens[b] / 64 + b, so that no table of chunks is needed.  floor(x / 64)
// + 1 never falls below the ceil((y - x) / 64) chunks of the tokens x .. y-1 by
// more than what floor(y / 64) makes up for, so ranges do not overlap.
inline int64_t max_chunks(int64_t total_tokens, int32_t batch) { return total_tokens / kChunk + batch; }

// Workspace bytes of one (chunk, value head).
size_t chunk_bytes(int rule, int dtype);

hipError_t launch_linear_prefill(const stepq_linear_desc& d, const LinearArgs& a, hipStream_t s);
hipError_t launch_linear_step(const stepq_linear_desc& d, const LinearArgs& a, hipStream_t s);

}  // namespace stepq
