// Host side of the verification of drafted tokens: argument checks, launches.  The
// operator is described in include/stepq_block.h.
#include "draft_internal.hpp"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMostRows = 1 << 22;    // a grid holds fewer than 2^32 threads; that many rows have a wave each

stepq_status check_sizes(int32_t batch, int32_t drafts, int32_t vocab) {
  if (batch < 0 || drafts < 0 || vocab < 1) return STEPQ_ERR_INVALID_ARG;
  if (drafts > stepq::kMostDrafts || vocab > 0x7fffffff - stepq::kVerifyTile) return STEPQ_ERR_UNSUPPORTED;
  return static_cast<int64_t>(batch) * (2 * drafts + 1) > kMostRows ? STEPQ_ERR_UNSUPPORTED : STEPQ_OK;
}

stepq_status from_hip(hipError_t e) { return e == hipSuccess ? STEPQ_OK : STEPQ_ERR_HIP; }

}  // namespace

extern "C" {

size_t stepq_verify_workspace_bytes(int32_t batch, int32_t drafts, int32_t vocab) {
  if (check_sizes(batch, drafts, vocab) != STEPQ_OK || batch == 0) return 0;
  return stepq::verify_workspace(batch, drafts, vocab).bytes;
}

stepq_status stepq_verify_drafts(int32_t batch, int32_t drafts, int32_t vocab, const void* logits, int32_t dtype,
                                 int64_t logits_stride, const void* draft_logits, int64_t draft_logits_stride,
                                 const int32_t* draft_tokens, const int32_t* num_drafts, const float* temperature,
                                 const float* uniforms, int32_t* accepted, int32_t* tokens, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const stepq_status st = check_sizes(batch, drafts, vocab);
  if (st != STEPQ_OK) return st;
  if (dtype != STEPQ_F32 && dtype != STEPQ_BF16 && dtype != STEPQ_F16) return STEPQ_ERR_INVALID_ARG;
  if (batch == 0) return STEPQ_OK;
  if (!logits || !uniforms || !accepted || !tokens || !workspace || (drafts > 0 && !draft_tokens)) return STEPQ_ERR_INVALID_ARG;
  const size_t e = dtype == STEPQ_F32 ? 4 : 2;
  const void* words[] = {draft_tokens, num_drafts, temperature, uniforms, accepted, tokens};
  for (const void* p : words)
    if (!aligned(p, 4)) return STEPQ_ERR_INVALID_ARG;
  if (!aligned(logits, e) || !aligned(draft_logits, e) || !aligned(workspace, 16)) return STEPQ_ERR_INVALID_ARG;
  if (logits_stride < vocab || (draft_logits && draft_logits_stride < vocab)) return STEPQ_ERR_INVALID_ARG;
  if (logits_stride > (int64_t{1} << 38) || draft_logits_stride > (int64_t{1} << 38)) return STEPQ_ERR_INVALID_ARG;
  const stepq::VerifyWorkspace w = stepq::verify_workspace(batch, drafts, vocab);
  if (workspace_bytes < w.bytes) return STEPQ_ERR_INVALID_ARG;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  stepq::VerifyArgs a{};
  a.logits = logits; a.draft_logits = drafts > 0 ? draft_logits : nullptr;
  a.logits_stride = logits_stride; a.draft_stride = draft_logits_stride;
  a.draft_tokens = draft_tokens; a.num_drafts = num_drafts; a.temperature = temperature; a.uniforms = uniforms;
  a.accepted = accepted; a.tokens = tokens;
  a.parts = reinterpret_cast<stepq::VerifyPart*>(base);
  a.plans = reinterpret_cast<stepq::VerifyPlan*>(base + w.plans);
  a.sums = reinterpret_cast<double*>(base + w.sums);
  a.batch = batch; a.drafts = drafts; a.vocab = vocab;
  a.num_parts = stepq::verify_parts(static_cast<int64_t>(batch) * (2 * drafts + 1), vocab);
  a.tiles = stepq::verify_tiles(vocab);
  a.part_tiles = (a.tiles + a.num_parts - 1) / a.num_parts;
  // a request's tiles go to workgroups of 4 waves, 1024 of them in all or a tile a wave
  int64_t groups = (1024 + batch - 1) / batch;
  if (groups > (a.tiles + 3) / 4) groups = (a.tiles + 3) / 4;
  a.groups = static_cast<int32_t>(groups);
  return from_hip(stepq::launch_verify(a, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
