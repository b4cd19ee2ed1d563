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

// A row's softmax: exp2((x - m) c) * scale; scale 0: everything is banned.
struct VerifyRow {
  double scale;
  float m;
  int32_t at;
};

// What a request's next token is drawn from.
struct VerifyPlan {
  VerifyRow p, q;
  int32_t n;          // drafts that are accepted
  int32_t minus;      // the token is drawn from p - q
  int32_t sharp;      // q is 1 at this token and nowhere else; -1: it is not
  int32_t pad;
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
  VerifyPlan* plans;             // [batch]
  int32_t batch;
  int32_t drafts;
  int32_t vocab;
  int32_t num_parts;             // waves a row is split over
  int32_t part_tiles;            // tiles of one part
  int32_t tiles;                 // of a row
  int32_t groups;                // workgroups that a request's tiles are split over
};

inline int32_t verify_tiles(int32_t vocab) { return (vocab + kVerifyTile - 1) / kVerifyTile; }

// Waves a row is split over: enough that all rows together give the chip 16384 of them (64 a compute
// unit, four times what it holds, since rows behind a request's drafts and greedy requests' leave waves without
// work), none of them shorter than a tile.  64 requests of up to 5 drafts over 131072 tokens, some greedy, us of the
// scan: with 4096 waves 85, with 16384 62.  us of calls with 4096, 8192, 16384 and 32768 waves where none is left out: 64 requests of
// 5 drafts over 131072 117, 108, 113, 114;  without draft logits 104, 69, 73, 75;  greedy 33, 25, 28, 33;  8 of 5 over 131072 39, 36, 36,
// 36;  16 of 4 over 32000 28, 26, 26, 26;  256 of 3 over 32000 80, 77, 81, 82.
inline int32_t verify_parts(int64_t rows, int32_t vocab) {
  int64_t parts = (16384 + rows - 1) / rows;
  if (parts > 64) parts = 64;
  const int32_t tiles = verify_tiles(vocab);
  return static_cast<int32_t>(parts > tiles ? tiles : parts);
}

struct VerifyWorkspace {
  size_t plans, sums, bytes;       // offsets; the parts are at 0
};
inline VerifyWorkspace verify_workspace(int32_t batch, int32_t drafts, int32_t vocab) {
  const int64_t rows = static_cast<int64_t>(batch) * (2 * drafts + 1);
  VerifyWorkspace w{};
  w.plans = static_cast<size_t>(rows) * verify_parts(rows, vocab) * sizeof(VerifyPart);
  w.sums = w.plans + static_cast<size_t>(batch) * sizeof(VerifyPlan);
  w.bytes = w.sums + static_cast<size_t>(batch) * verify_tiles(vocab) * 2 * sizeof(double);
  return w;
}

hipError_t launch_verify(const VerifyArgs& a, int dtype, hipStream_t s);

}  // namespace stepq
