// Internal declarations shared by the host API (norm_api.cpp) and the gfx950
// kernels (norm_kernels.hip) of the norms around a block.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/stepq_block.h"

namespace stepq {

constexpr int kMostWidth = 16384;

// A tensor of tokens; nullptr: none.
struct NormRows {
  const void* p;
  int64_t stride;        // elements from token to token
};

struct NormArgs {
  NormRows block, gate, residual;       // read
  NormRows out, normed;                 // forward: written; backward: out is read
  NormRows d_out, d_normed;             // backward, read
  NormRows d_block, d_gate, d_residual; // backward, written
  const float* post_weight;
  const float* scale;
  const float* pre_weight;
  float* d_post_weight;
  float* d_scale;
  float* d_pre_weight;
  float* partial;                       // [3][groups][width]
  int32_t rows;                         // tokens * heads
  int32_t heads;
  int32_t width;
  int32_t groups;
  int32_t post;
  int32_t pre;
  int32_t silu;
  float eps;
};

// Lanes that share a row and the 16-byte pieces each of them holds.
struct NormShape {
  int lanes, pieces;
};
inline NormShape norm_shape(int width, int dtype, bool backward) {
  const int n = dtype == STEPQ_F32 ? (width + 3) / 4 : (width + 7) / 8;      // pieces of a row
  if (n <= 4) return {4, 1};
  if (n <= 16) return {16, 1};
  if (n <= 64) return {64, 1};
  if (n <= 128) return {128, 1};
  if (n <= 256) return {256, 1};
  if (n <= 512) return {512, 1};
  // a backward pass needs more registers than the 128 that each of 1024 lanes has: 4096 tokens of 8192 bfloat16
  // values, 266 us with 1024 lanes, 155 with 512; binary32 271, 213
  if (backward && dtype != STEPQ_F32 && n <= 1024) return {512, 2};
  if (backward && dtype == STEPQ_F32 && n > 1024 && n <= 2048) return {512, 4};
  if (n <= 1024) return {1024, 1};
  return {1024, n <= 2048 ? 2 : 4};
}

// Rows that a workgroup has under way at a time.
constexpr int kNormThreads = 256;
inline int norm_rows_at_once(const NormShape& s) { return s.lanes < kNormThreads ? kNormThreads / s.lanes : 1; }

// Workgroups of a backward pass, each with its part of the weights' gradients: as many as the chip holds at
// once with 150 to 160 registers a lane.  8192 tokens of 4096 with 256 workgroups of 512 lanes 127 us, with 512 146
// (half as many registers, to hold two of them a compute unit: 307, by what goes to memory and back).
inline int32_t norm_groups(const stepq_norm_desc& d, int64_t rows) {
  const NormShape s = norm_shape(d.width, d.dtype, true);
  const int at_once = norm_rows_at_once(s);
  const int64_t all = (rows + at_once - 1) / at_once, most = s.lanes > kNormThreads ? 256 : 768;
  return static_cast<int32_t>(all < most ? all : most);
}

hipError_t launch_norm_forward(const NormArgs& a, int dtype, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs& a, int dtype, hipStream_t s);

}  // namespace stepq
