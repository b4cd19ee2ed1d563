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
  uint32_t* ticket;            // see scan_workspace
  uint64_t* ends;
  uint64_t* links;
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

struct ScanWorkspace {
  size_t ends, links, partial, bytes;     // offsets; the ticket is at 0
};
inline ScanWorkspace scan_workspace(const stepq_scan_desc& d, int64_t total_tokens, int64_t batch, bool backward) {
  const size_t n = static_cast<size_t>(scan_pieces(total_tokens, batch)) * d.width;
  const size_t words = scan_linked(total_tokens) ? (n * 8 + 15) / 16 * 16 : 0;
  ScanWorkspace w{};
  w.ends = words ? 16 : 0;
  w.links = w.ends + words;
  w.partial = w.links + words;
  w.bytes = w.partial + (backward ? (n * 4 + 15) / 16 * 16 : 0);
  return w;
}

hipError_t launch_scan_forward(const ScanArgs& a, int dtype, hipStream_t s);
hipError_t launch_scan_backward(const ScanArgs& a, int dtype, hipStream_t s);
hipError_t launch_scan_step(const ScanArgs& a, int dtype, hipStream_t s);

}  // namespace stepq
