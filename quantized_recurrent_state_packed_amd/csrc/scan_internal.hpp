// Internal declarations shared by the host API (scan_api.cpp) and the gfx950
// kernels (scan_kernels.hip) of the gated linear recurrence.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/stepq_block.h"

namespace stepq {

// Tokens that a wave holds, and waves of a workgroup, one behind the other in time.  us of a prompt of
// 32768 tokens x 4096 bfloat16 channels, of 8 prompts of 8192 x 6144:
//   16 tokens of 4 waves 300, 116;  16 of 8 253, 107;  16 of 16 324, 138;  32 of 4 238, 105;  32 of 8 271, 117
// The backward pass holds twice the tensors: us of forward and backward of 12288 tokens x 4096 with 8 tokens of
// 4 waves 345, of 6 422, of 8 300, of 16 446; 16 tokens of 4 waves 390.
constexpr int kScanTokens = 32, kScanWaves = 4;
constexpr int kBackTokens = 8, kBackWaves = 8;
constexpr int kFewTokens = 8, kFewWaves = 8;
constexpr int kScanPiece = kScanTokens * kScanWaves;      // tokens of a workgroup
constexpr int kBackPiece = kBackTokens * kBackWaves;
constexpr int kFewPiece = kFewTokens * kFewWaves;
static_assert(kScanTokens % kBackTokens == 0 && kFewTokens % kBackTokens == 0);      // a forward pass saves a state every kBackTokens tokens

struct ScanArgs {
  const void* x;
  const void* ga;
  const void* gx;
  const void* dy;              // backward only
  int64_t x_stride;            // elements from token to token
  int64_t ga_stride;
  int64_t gx_stride;
  int64_t dy_stride;
  const float* decay;
  const int32_t* cu_seqlens;   // nullptr: single tokens
  const int32_t* slot_ids;     // nullptr: no states
  const uint8_t* resume;       // nullptr: all from zero
  float* state;                // backward: the states' gradients
  void* y;                     // backward: dx
  void* dga;                   // backward only
  void* dgx;
  int64_t y_stride;
  int64_t dga_stride;
  int64_t dgx_stride;
  float* saved;                // nullptr: nothing is saved
  float* ddecay;
  float* partial;              // backward: every piece's part of ddecay
  uint32_t* ticket;            // nullptr: no request is longer than a piece; see ScanWorkspace
  uint64_t* maps;
  uint64_t* ends;
  float* speeds;
  int64_t words;               // of 16 bytes, to be set before the pieces run
  int64_t total_tokens;
  int32_t batch;
  int32_t num_slots;
  int32_t width;
  int32_t blocks;              // workgroups that a piece's channels take
  uint32_t pieces;
  float rate;
  int32_t piece;               // tokens of a piece
};

// Pieces of `piece` tokens of all requests together: request b's start at index
// cu_seqlens[b] / piece + b, so that no table of them is needed.  From b to b + 1 the index grows by
// at least the ceil((cu[b + 1] - cu[b]) / piece) pieces of request b, and by 1 for an empty one.
inline int64_t scan_pieces(int64_t total_tokens, int64_t batch, int piece) { return total_tokens / piece + batch; }

// Tokens of a piece.  A forward pass of fewer workgroups than fill the chip takes smaller pieces, of more waves that have fewer
// tokens each to go through.  us of bfloat16 calls, 128 tokens a piece (32 of 4 waves) against 64 (8 of 8), by workgroups
// of the former, counted with 128 channels each (binary32 and odd rows have 64 in one, and twice as many): 37 tokens x 4096 (32) 8.2 : 5.2;  200 x 4096 (64) 12.5 : 10.4;  20000 x 128 (157) 26.2 : 23.8;  700 x 4096 (192)
// 15.6 : 16.8;  1400 x 4096 (352) 23.7 : 24.8;  2800 x 4096 (704) 36.6 : 38.0;  5 prompts of 3001 x 1001 binary32 (224) 20 : 24.5.
constexpr int64_t kFewGroups = 160;
inline int scan_piece(const stepq_scan_desc& d, int64_t total_tokens, int64_t batch, bool backward) {
  if (backward) return kBackPiece;
  return scan_pieces(total_tokens, batch, kScanPiece) * ((d.width + 127) / 128) < kFewGroups ? kFewPiece : kScanPiece;
}

// What a call over requests longer than a piece keeps in its workspace: a ticket (at 0), every
// piece's map of the state before it to the state behind it, the states behind pieces, each
// channel's logarithm of the retention at an open gate; and a backward pass every piece's part
// of ddecay.  Offsets in bytes.
struct ScanWorkspace {
  size_t maps, ends, speeds, partial, bytes;
};
inline ScanWorkspace scan_workspace(const stepq_scan_desc& d, int64_t total_tokens, int64_t batch, bool backward) {
  const auto whole = [](size_t bytes) { return (bytes + 15) / 16 * 16; };
  const int piece = scan_piece(d, total_tokens, batch, backward);
  const size_t n = static_cast<size_t>(scan_pieces(total_tokens, batch, piece)) * d.width;
  const bool linked = total_tokens > piece;      // requests of a piece or less have nothing to hand on
  ScanWorkspace w{};
  w.maps = linked ? 16 : 0;
  w.ends = w.maps + (linked ? whole(n * 8) : 0);
  w.speeds = w.ends + (linked ? whole(n * 8) : 0);
  w.partial = w.speeds + (linked ? whole(static_cast<size_t>(d.width) * 4) : 0);
  w.bytes = w.partial + (backward ? whole(n * 4) : 0);
  return w;
}

// Saved: the states before every kBackTokens tokens, by the same index rule.
inline size_t scan_saved(const stepq_scan_desc& d, int64_t total_tokens, int64_t batch) {
  return static_cast<size_t>(scan_pieces(total_tokens, batch, kBackTokens)) * d.width * sizeof(float);
}

hipError_t launch_scan_forward(const ScanArgs& a, int dtype, hipStream_t s);
hipError_t launch_scan_backward(const ScanArgs& a, int dtype, hipStream_t s);
hipError_t launch_scan_step(const ScanArgs& a, int dtype, hipStream_t s);

}  // namespace stepq
