// Internal declarations shared by the host API (beam_api.cpp) and the gfx950
// kernels (beam_kernels.hip) of beam selection and state reordering.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/stepq_seq.h"

namespace stepq {

constexpr int kMaxBeams = 64;      // beams of a request, and candidates: one wave holds a list of either
constexpr int kTile = 1024;        // logits one wave holds at a time

struct SelectArgs {
  const void* logits;
  int64_t stride;            // elements from row to row
  const float* scores;
  const uint8_t* finished;   // nullptr: none
  int32_t* tokens;
  int32_t* parents;
  float* out_scores;
  uint8_t* workspace;
  int32_t batch;
  int32_t beams;
  int32_t vocab;
  int32_t num_out;
  int32_t eos;
  int32_t parts;             // waves a row is split over
  int32_t tiles;             // tiles of one part
};

// Waves a row's logits are split over: enough that all rows together give the
// chip kScanWaves waves, none of them shorter than a tile.
int select_parts(int64_t rows, int32_t vocab);

__host__ __device__ inline size_t select_part_bytes(int32_t num_out) {
  return sizeof(float) * (2 + 2 * static_cast<size_t>(num_out));
}

struct ReorderArgs {
  const int32_t* slot_ids;
  const int32_t* parents;
  int32_t* new_slot_ids;
  int32_t beams;
  int32_t num_slots;
  int32_t num_regions;
  struct {
    uint8_t* base;
    uint64_t slot_bytes;
    uint32_t first_segment;  // segments of the regions before this one
  } regions[STEPQ_MAX_REGIONS];
};

constexpr int kSegment = 32768;    // bytes of a slot that one workgroup copies

hipError_t launch_beam_select(const SelectArgs& a, int dtype, hipStream_t s);
hipError_t launch_beam_reorder(const ReorderArgs& a, int32_t batch, uint32_t segments, hipStream_t s);

}  // namespace stepq
