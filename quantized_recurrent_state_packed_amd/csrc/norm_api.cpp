// Host side of the norms around a block: argument checks, launches.  The operators
// are described in include/stepq_block.h.
#include "norm_internal.hpp"

#include <cmath>

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

stepq_status check_sizes(const stepq_norm_desc* d, int64_t tokens) {
  if (!d || d->width < 1 || d->heads < 1) return STEPQ_ERR_INVALID_ARG;
  if (d->dtype != STEPQ_F32 && d->dtype != STEPQ_BF16 && d->dtype != STEPQ_F16) return STEPQ_ERR_INVALID_ARG;
  if (d->activation != STEPQ_GATE_SILU && d->activation != STEPQ_GATE_SIGMOID) return STEPQ_ERR_INVALID_ARG;
  if ((d->post != 0 && d->post != 1) || (d->pre != 0 && d->pre != 1)) return STEPQ_ERR_INVALID_ARG;
  if (!std::isnormal(d->eps) || d->eps < 0.0f || tokens < 0) return STEPQ_ERR_INVALID_ARG;
  if (d->width > stepq::kMostWidth) return STEPQ_ERR_UNSUPPORTED;
  return tokens > 0x7fffffffLL / d->heads ? STEPQ_ERR_UNSUPPORTED : STEPQ_OK;
}

int elem_bytes(int dtype) { return dtype == STEPQ_F32 ? 4 : 2; }

bool rows_ok(const stepq::NormRows& r, const stepq_norm_desc& d) {
  return aligned(r.p, elem_bytes(d.dtype)) && r.stride >= static_cast<int64_t>(d.heads) * d.width &&
         r.stride <= (int64_t{1} << 40);
}

// An output in an input's buffer overwrites what its own lanes have read, if the rows lie alike.
bool apart_or_alike(const stepq::NormRows& out, const stepq::NormRows& in, int64_t tokens) {
  return !out.p || out.p != in.p || out.stride == in.stride || tokens == 1;
}

stepq_status from_hip(hipError_t e) { return e == hipSuccess ? STEPQ_OK : STEPQ_ERR_HIP; }

// What both passes share.
stepq::NormArgs arguments(const stepq_norm_desc& d, int64_t tokens) {
  stepq::NormArgs a{};
  a.rows = static_cast<int32_t>(tokens * d.heads);
  a.heads = d.heads; a.width = d.width;
  a.post = d.post; a.pre = d.pre; a.silu = d.activation == STEPQ_GATE_SILU; a.eps = d.eps;
  return a;
}

// Rows of all tokens at one distance are rows of tokens of one head.
void flatten(stepq::NormArgs& a) {
  if (a.heads == 1) return;
  stepq::NormRows* all[] = {&a.block, &a.gate, &a.residual, &a.out, &a.normed, &a.d_out, &a.d_normed, &a.d_block, &a.d_gate,
                            &a.d_residual};
  for (const stepq::NormRows* r : all)
    if (r->p && r->stride != static_cast<int64_t>(a.heads) * a.width) return;
  for (stepq::NormRows* r : all) r->stride = a.width;
  a.heads = 1;
}

}  // namespace

extern "C" {

stepq_status stepq_norm_forward(const stepq_norm_desc* d, int64_t tokens, const void* block, int64_t block_stride,
                                const void* gate, int64_t gate_stride, const void* residual, int64_t residual_stride,
                                const float* post_weight, const float* scale, const float* pre_weight, void* out,
                                int64_t out_stride, void* normed, int64_t normed_stride, void* stream) {
  const stepq_status st = check_sizes(d, tokens);
  if (st != STEPQ_OK) return st;
  if (tokens == 0) return STEPQ_OK;
  if (!block || (!out && !d->pre) || (normed != nullptr) != (d->pre != 0) || (post_weight && !d->post) ||
      (pre_weight && !d->pre) || out == normed)
    return STEPQ_ERR_INVALID_ARG;
  stepq::NormArgs a = arguments(*d, tokens);
  a.block = {block, block_stride};
  a.gate = {gate, gate_stride};
  a.residual = {residual, residual_stride};
  a.out = {out, out_stride};
  a.normed = {normed, normed_stride};
  const stepq::NormRows* rows[] = {&a.block, &a.gate, &a.residual, &a.out, &a.normed};
  for (const stepq::NormRows* r : rows)
    if (r->p && !rows_ok(*r, *d)) return STEPQ_ERR_INVALID_ARG;
  for (const stepq::NormRows* to : {&a.out, &a.normed})
    for (const stepq::NormRows* from : {&a.block, &a.gate, &a.residual})
      if (!apart_or_alike(*to, *from, tokens)) return STEPQ_ERR_INVALID_ARG;
  if (!aligned(post_weight, 4) || !aligned(scale, 4) || !aligned(pre_weight, 4)) return STEPQ_ERR_INVALID_ARG;
  a.post_weight = post_weight; a.scale = scale; a.pre_weight = pre_weight;
  flatten(a);
  return from_hip(stepq::launch_norm_forward(a, d->dtype, static_cast<hipStream_t>(stream)));
}

size_t stepq_norm_workspace_bytes(const stepq_norm_desc* d, int64_t tokens) {
  if (check_sizes(d, tokens) != STEPQ_OK) return 0;
  return sizeof(float) * 3 * static_cast<size_t>(stepq::norm_groups(*d, tokens * d->heads)) * d->width;
}

stepq_status stepq_norm_backward(const stepq_norm_desc* d, int64_t tokens, const void* block, int64_t block_stride,
                                 const void* gate, int64_t gate_stride, const void* out, int64_t out_stride,
                                 const float* post_weight, const float* scale, const float* pre_weight, const void* d_out,
                                 int64_t d_out_stride, const void* d_normed, int64_t d_normed_stride, void* d_block,
                                 int64_t d_block_stride, void* d_gate, int64_t d_gate_stride, void* d_residual,
                                 int64_t d_residual_stride, float* d_post_weight, float* d_scale, float* d_pre_weight,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  const stepq_status st = check_sizes(d, tokens);
  if (st != STEPQ_OK) return st;
  if ((post_weight && !d->post) || (pre_weight && !d->pre) || (d_post_weight && !post_weight) || (d_scale && !scale) ||
      (d_pre_weight && !pre_weight))
    return STEPQ_ERR_INVALID_ARG;
  const void* floats[] = {post_weight, scale, pre_weight, d_post_weight, d_scale, d_pre_weight};
  for (const void* p : floats)
    if (!aligned(p, 4)) return STEPQ_ERR_INVALID_ARG;
  stepq::NormArgs a = arguments(*d, tokens);
  a.post_weight = post_weight; a.scale = scale; a.pre_weight = pre_weight;
  a.d_post_weight = d_post_weight; a.d_scale = d_scale; a.d_pre_weight = d_pre_weight;
  if (tokens > 0) {
    if (!block || !d_block || (gate != nullptr) != (d_gate != nullptr) || (d_normed != nullptr) != (d->pre != 0) ||
        (d->pre ? !out : !d_out))
      return STEPQ_ERR_INVALID_ARG;
    if (d_block == d_gate || d_block == d_residual || (d_gate && d_gate == d_residual)) return STEPQ_ERR_INVALID_ARG;
    a.block = {block, block_stride};
    a.gate = {gate, gate_stride};
    a.out = {d->pre ? out : nullptr, out_stride};
    a.d_out = {d_out, d_out_stride};
    a.d_normed = {d_normed, d_normed_stride};
    a.d_block = {d_block, d_block_stride};
    a.d_gate = {d_gate, d_gate_stride};
    a.d_residual = {d_residual, d_residual_stride};
    const stepq::NormRows* rows[] = {&a.block, &a.gate, &a.out, &a.d_out, &a.d_normed, &a.d_block, &a.d_gate, &a.d_residual};
    for (const stepq::NormRows* r : rows)
      if (r->p && !rows_ok(*r, *d)) return STEPQ_ERR_INVALID_ARG;
    for (const stepq::NormRows* to : {&a.d_block, &a.d_gate, &a.d_residual})
      for (const stepq::NormRows* from : {&a.block, &a.gate, &a.out, &a.d_out, &a.d_normed})
        if (!apart_or_alike(*to, *from, tokens)) return STEPQ_ERR_INVALID_ARG;
    if (d_post_weight || d_scale || d_pre_weight) {
      if (!workspace || !aligned(workspace, 16) || workspace_bytes < stepq_norm_workspace_bytes(d, tokens))
        return STEPQ_ERR_INVALID_ARG;
      a.partial = static_cast<float*>(workspace);
    }
    a.groups = stepq::norm_groups(*d, a.rows);
    flatten(a);
  }
  return from_hip(stepq::launch_norm_backward(a, d->dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
