// Internal declarations shared by the host API (scan_api.cpp) and the gfx950
// kernels (scan_kernels.hip) of the gated linear recurrence.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/stepq_block.h"

namespace stepq {

constexpr int kScanTokens = 8;                            // tokens a wave holds
constexpr int kScanRows = 8;                              // waves of a workgroup, one behind the other in time
constexpr int kPiece = kScanTokens * kScanRows;           // tokens of a workgroup

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
};

// Pieces of all requests together: request b's start at index cu_seqlens[b] / kPiece + b, so
// that no table of them is needed.  From b to b + 1 the index grows by at least the
// ceil((cu[b + 1] - cu[b]) / kPiece) pieces of request b, and by 1 for an empty one.
inline int64_t scan_pieces(int64_t total_tokens, int64_t batch) { return total_tokens / kPiece + batch; }

// Requests of a piece or less have nothing to hand on.
inline bool scan_linked(int64_t total_tokens) { return total_tokens > kPiece; }

// What a call over requests longer than a piece keeps in its workspace: a ticket (at 0), every
// piece's map of the state before it to the state behind it, the states behind pieces, each
// channel's logarithm of the retention at an open gate; and a backward pass every piece's part
// of ddecay.  Offsets in bytes.
struct ScanWorkspace {
  size_t maps, ends, speeds, partial, bytes;
};
inline ScanWorkspace scan_workspace(const stepq_scan_desc& d, int64_t total_tokens, int64_t batch, bool backward) {
  const auto whole = [](size_t bytes) { return (bytes + 15) / 16 * 16; };
  const size_t n = static_cast<size_t>(scan_pieces(total_tokens, batch)) * d.width;
  const bool linked = scan_linked(total_tokens);
  ScanWorkspace w{};
  w.maps = linked ? 16 : 0;
  w.ends = w.maps + (linked ? whole(n * 8) : 0);
  w.speeds = w.ends + (linked ? whole(n * 8) : 0);
  w.partial = w.speeds + (linked ? whole(static_cast<size_t>(d.width) * 4) : 0);
  w.bytes = w.partial + (backward ? whole(n * 4) : 0);
  return w;
}

hipError_t launch_scan_forward(const ScanArgs& a, int dtype, hipStream_t s);
hipError_t launch_scan_backward(const ScanArgs& a, int dtype, hipStream_t s);
hipError_t launch_scan_step(const ScanArgs& a, int dtype, hipStream_t s);

}  // namespace stepq
