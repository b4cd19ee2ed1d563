// Internal declarations shared by the host API (draft_api.cpp) and the gfx950
// kernels (draft_kernels.hip) of the verification of drafted tokens.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/stepq_block.h"

namespace stepq {

constexpr int kMostDrafts = 63;        // a wave holds a request's rows
constexpr int kVerifyTile = 1024;      // logits a wave holds at a time

// What a wave found in its part of a row: sum of exp2((x - m) c) over it, and for greedy
// requests the largest logit and its place.
struct VerifyPart {
  double sum;
  float m;
  int32_t at;
};

struct VerifyArgs {
  const void* logits;
  const void* draft_logits;      // nullptr: the draft was certain
  int64_t logits_stride;         // elements from row to row
  int64_t draft_stride;
  const int32_t* draft_tokens;
  const int32_t* num_drafts;     // nullptr: all
  const float* temperature;      // nullptr: 1
  const float* uniforms;
  int32_t* accepted;
  int32_t* tokens;
  VerifyPart* parts;             // [batch][2 drafts + 1][num_parts], the target's rows first
  double* sums;                  // [batch][tiles][2]: of max(p - q, 0) and of p over a tile
  uint32_t* arrived;             // [batch]
  int32_t batch;
  int32_t drafts;
  int32_t vocab;
  int32_t num_parts;             // waves a row is split over
  int32_t part_tiles;            // tiles of one part
  int32_t tiles;                 // of a row
  int32_t pick_groups;           // workgroups that a request's tiles are split over
};

inline int32_t verify_tiles(int32_t vocab) { return (vocab + kVerifyTile - 1) / kVerifyTile; }

// Waves a row is split over: enough that all rows together give the chip 4096 of them (16 a
// compute unit), none of them shorter than a tile.
inline int32_t verify_parts(int64_t rows, int32_t vocab) {
  int64_t parts = (4096 + rows - 1) / rows;
  if (parts > 64) parts = 64;
  const int32_t tiles = verify_tiles(vocab);
  return static_cast<int32_t>(parts > tiles ? tiles : parts);
}

struct VerifyWorkspace {
  size_t sums, arrived, bytes;       // offsets; the parts are at 0
};
inline VerifyWorkspace verify_workspace(int32_t batch, int32_t drafts, int32_t vocab) {
  const int64_t rows = static_cast<int64_t>(batch) * (2 * drafts + 1);
  VerifyWorkspace w{};
  w.sums = static_cast<size_t>(rows) * verify_parts(rows, vocab) * sizeof(VerifyPart);
  w.arrived = w.sums + static_cast<size_t>(batch) * verify_tiles(vocab) * 2 * sizeof(double);
  w.bytes = w.arrived + (static_cast<size_t>(batch) * sizeof(uint32_t) + 15) / 16 * 16;
  return w;
}

hipError_t launch_verify(const VerifyArgs& a, int dtype, hipStream_t s);

}  // namespace stepq
