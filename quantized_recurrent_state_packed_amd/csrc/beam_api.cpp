// Host side of beam selection and state reordering: argument checks, launches.
// The operators are described in include/stepq_seq.h.
#include "beam_internal.hpp"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMostRows = 1 << 23;    // beams of a call: a grid holds fewer than 2^32 threads

stepq_status check_sizes(int32_t batch, int32_t beams, int32_t vocab, int32_t num_out) {
  if (batch < 0 || beams < 1 || vocab < 1 || num_out < 1) return STEPQ_ERR_INVALID_ARG;
  if (beams > stepq::kMaxBeams || num_out > 64) return STEPQ_ERR_UNSUPPORTED;
  if (vocab > 0x7fffffff - stepq::kTile) return STEPQ_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(batch) * beams > kMostRows) return STEPQ_ERR_UNSUPPORTED;
  return STEPQ_OK;
}

stepq_status from_hip(hipError_t e) { return e == hipSuccess ? STEPQ_OK : STEPQ_ERR_HIP; }

}  // namespace

extern "C" {

size_t stepq_beam_workspace_bytes(int32_t batch, int32_t beams, int32_t vocab, int32_t num_out) {
  if (check_sizes(batch, beams, vocab, num_out) != STEPQ_OK) return 0;
  const int64_t rows = static_cast<int64_t>(batch) * beams;
  return static_cast<size_t>(rows) * stepq::select_parts(rows, vocab) * stepq::select_part_bytes(num_out);
}

stepq_status stepq_beam_select(int32_t batch, int32_t beams, int32_t vocab, int32_t num_out,
                               const void* logits, int32_t dtype, int64_t logits_stride, const float* scores,
                               const uint8_t* finished, int32_t eos_token, int32_t* tokens, int32_t* parents,
                               float* out_scores, void* workspace, size_t workspace_bytes, void* stream) {
  const stepq_status st = check_sizes(batch, beams, vocab, num_out);
  if (st != STEPQ_OK) return st;
  if (dtype != STEPQ_F32 && dtype != STEPQ_BF16 && dtype != STEPQ_F16) return STEPQ_ERR_INVALID_ARG;
  if (batch == 0) return STEPQ_OK;
  if (!logits || !scores || !tokens || !parents || !out_scores || !workspace) return STEPQ_ERR_INVALID_ARG;
  const size_t e = dtype == STEPQ_F32 ? 4 : 2;
  if (!aligned(logits, e) || !aligned(workspace, 16) || !aligned(scores, 4) || !aligned(tokens, 4) ||
      !aligned(parents, 4) || !aligned(out_scores, 4))
    return STEPQ_ERR_INVALID_ARG;
  if (logits_stride < vocab) return STEPQ_ERR_INVALID_ARG;
  if (workspace_bytes < stepq_beam_workspace_bytes(batch, beams, vocab, num_out)) return STEPQ_ERR_INVALID_ARG;
  stepq::SelectArgs a{};
  a.logits = logits;
  a.stride = logits_stride;
  a.scores = scores;
  a.finished = finished;
  a.tokens = tokens;
  a.parents = parents;
  a.out_scores = out_scores;
  a.workspace = static_cast<uint8_t*>(workspace);
  a.batch = batch;
  a.beams = beams;
  a.vocab = vocab;
  a.num_out = num_out;
  a.eos = eos_token;
  a.parts = stepq::select_parts(static_cast<int64_t>(batch) * beams, vocab);
  // a row is read from the 16-byte boundary at or below its start
  const int64_t all = (static_cast<int64_t>(vocab) + static_cast<int64_t>(16 / e) - 1 + stepq::kTile - 1) / stepq::kTile;
  a.tiles = static_cast<int32_t>((all + a.parts - 1) / a.parts);
  return from_hip(stepq::launch_beam_select(a, dtype, static_cast<hipStream_t>(stream)));
}

stepq_status stepq_beam_reorder(int32_t batch, int32_t beams, const int32_t* slot_ids, const int32_t* parents,
                                int32_t num_slots, const stepq_region* regions, int32_t num_regions,
                                int32_t* new_slot_ids, void* stream) {
  if (batch < 0 || beams < 1 || num_slots < 1 || num_regions < 0) return STEPQ_ERR_INVALID_ARG;
  if (beams > stepq::kMaxBeams || num_regions > STEPQ_MAX_REGIONS) return STEPQ_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(batch) * beams > kMostRows) return STEPQ_ERR_UNSUPPORTED;
  if (batch == 0) return STEPQ_OK;
  if (!slot_ids || !parents || !new_slot_ids || (num_regions > 0 && !regions)) return STEPQ_ERR_INVALID_ARG;
  if (!aligned(slot_ids, 4) || !aligned(parents, 4) || !aligned(new_slot_ids, 4)) return STEPQ_ERR_INVALID_ARG;
  if (new_slot_ids == slot_ids || new_slot_ids == parents) return STEPQ_ERR_INVALID_ARG;
  stepq::ReorderArgs a{};
  a.slot_ids = slot_ids;
  a.parents = parents;
  a.new_slot_ids = new_slot_ids;
  a.beams = beams;
  a.num_slots = num_slots;
  a.num_regions = num_regions;
  uint64_t segments = 0;
  for (int i = 0; i < num_regions; ++i) {
    const stepq_region& r = regions[i];
    if (!r.base || !aligned(r.base, 16) || r.slot_bytes == 0 || r.slot_bytes % 16 != 0) return STEPQ_ERR_INVALID_ARG;
    a.regions[i].base = static_cast<uint8_t*>(r.base);
    a.regions[i].slot_bytes = r.slot_bytes;
    a.regions[i].first_segment = static_cast<uint32_t>(segments);
    segments += (r.slot_bytes + stepq::kSegment - 1) / stepq::kSegment;
    if (segments > 65535) return STEPQ_ERR_UNSUPPORTED;   // the grid's second dimension
  }
  return from_hip(stepq::launch_beam_reorder(a, batch, static_cast<uint32_t>(segments == 0 ? 1 : segments),
                                             static_cast<hipStream_t>(stream)));
}

}  // extern "C"
