// Host side of the linear-attention entry points: argument checks, launches.
// The operators are described in include/stepq_seq.h.
#include "linear_internal.hpp"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMostHeads = (1 << 23) - 1;        // (request, head) pairs of a call
constexpr int64_t kMostChunkHeads = (1 << 24) - 1;   // (chunk, head) pairs of a call

int elem_bytes(int dtype) { return dtype == STEPQ_F32 ? 4 : 2; }

stepq_status check_desc(const stepq_linear_desc* d) {
  if (!d || d->num_heads < 1 || d->num_qk_heads < 1 || d->d < 1) return STEPQ_ERR_INVALID_ARG;
  if (d->rule != STEPQ_RULE_ADDITIVE && d->rule != STEPQ_RULE_DELTA) return STEPQ_ERR_INVALID_ARG;
  if (d->dtype != STEPQ_F32 && d->dtype != STEPQ_BF16 && d->dtype != STEPQ_F16) return STEPQ_ERR_INVALID_ARG;
  if (d->num_heads % d->num_qk_heads != 0) return STEPQ_ERR_INVALID_ARG;
  if (!(d->d == 16 || d->d == 32 || d->d == 64 || d->d == 128)) return STEPQ_ERR_UNSUPPORTED;
  if (d->num_heads > (1 << 16)) return STEPQ_ERR_UNSUPPORTED;
  return STEPQ_OK;
}

// A token's stride: room for its heads, whole 16-byte units.
bool stride_ok(int64_t stride, int64_t row, int esize) { return stride >= row && (stride * esize) % 16 == 0; }

stepq_status check_tensors(const stepq_linear_desc& d, const void* q, int64_t qs, const void* k, int64_t ks,
                           const void* v, int64_t vs, const float* beta, const float* gate, const float* state,
                           const void* o, int64_t os) {
  if (!q || !k || !v || !gate || !state || !o) return STEPQ_ERR_INVALID_ARG;
  if ((d.rule == STEPQ_RULE_DELTA) != (beta != nullptr)) return STEPQ_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, state, o};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return STEPQ_ERR_INVALID_ARG;
  if (!aligned(beta, 4) || !aligned(gate, 4)) return STEPQ_ERR_INVALID_ARG;
  const int e = elem_bytes(d.dtype);
  const int64_t qk = static_cast<int64_t>(d.num_qk_heads) * d.d, vo = static_cast<int64_t>(d.num_heads) * d.d;
  if (!stride_ok(qs, qk, e) || !stride_ok(ks, qk, e) || !stride_ok(vs, vo, e) || !stride_ok(os, vo, e))
    return STEPQ_ERR_INVALID_ARG;
  const int64_t most = 1 << 24;     // a chunk's 64 rows are addressed in 32 bits
  return qs <= most && ks <= most && vs <= most && os <= most ? STEPQ_OK : STEPQ_ERR_UNSUPPORTED;
}

stepq_status from_hip(hipError_t e) { return e == hipSuccess ? STEPQ_OK : STEPQ_ERR_HIP; }

}  // namespace

extern "C" {

size_t stepq_linear_workspace_bytes(const stepq_linear_desc* d, int32_t batch, int64_t total_tokens) {
  if (check_desc(d) != STEPQ_OK || batch < 0 || total_tokens < 0 || total_tokens > 0x7fffffffLL) return 0;
  return stepq::most_workspace(*d, total_tokens, batch);
}

size_t stepq_linear_prefill_bytes(const stepq_linear_desc* d, int32_t batch, int64_t total_tokens) {
  if (check_desc(d) != STEPQ_OK || batch < 1 || total_tokens < 0 || total_tokens > 0x7fffffffLL) return 0;
  return stepq::call_workspace(*d, total_tokens, batch);
}

stepq_status stepq_linear_prefill(const stepq_linear_desc* d, int32_t batch, int64_t total_tokens,
                                  const int32_t* cu_seqlens, const void* q, int64_t q_stride, const void* k,
                                  int64_t k_stride, const void* v, int64_t v_stride, const float* beta,
                                  const float* gate, const int32_t* slot_ids, int32_t num_slots,
                                  const uint8_t* resume, float* state, void* o, int64_t o_stride,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  stepq_status st = check_desc(d);
  if (st != STEPQ_OK) return st;
  if (batch < 0 || total_tokens < 0 || num_slots < 1) return STEPQ_ERR_INVALID_ARG;
  if (batch == 0) return STEPQ_OK;
  if (!cu_seqlens || !slot_ids || !aligned(cu_seqlens, 4) || !aligned(slot_ids, 4))
    return STEPQ_ERR_INVALID_ARG;
  // int32 cu_seqlens; grids of fewer than 2^32 threads: 256 for every (chunk, head), up to
  // 512 for every (request, head)
  if (total_tokens > 0x7fffffffLL) return STEPQ_ERR_UNSUPPORTED;
  if (stepq::max_chunks(total_tokens, batch) > kMostChunkHeads / d->num_heads) return STEPQ_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(batch) * d->num_heads > kMostHeads) return STEPQ_ERR_UNSUPPORTED;
  st = check_tensors(*d, q, q_stride, k, k_stride, v, v_stride, beta, gate, state, o, o_stride);
  if (st != STEPQ_OK) return st;
  const size_t need = stepq::call_workspace(*d, total_tokens, batch);
  if ((need > 0 && !workspace) || !aligned(workspace, 16) || workspace_bytes < need) return STEPQ_ERR_INVALID_ARG;
  stepq::LinearArgs a{};
  a.q = q; a.k = k; a.v = v;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.beta = beta; a.gate = gate;
  a.slot_ids = slot_ids; a.cu_seqlens = cu_seqlens; a.resume = resume;
  a.state = state; a.o = o; a.o_stride = o_stride;
  a.total_tokens = total_tokens; a.batch = batch; a.num_slots = num_slots;
  a.H = d->num_heads; a.rep = d->num_heads / d->num_qk_heads;
  a.workspace = static_cast<uint8_t*>(workspace);
  a.segment = stepq::segment_chunks(*d, total_tokens, batch);
  a.apart = stepq::chunks_apart(*d, total_tokens, batch);
  return from_hip(stepq::launch_linear_prefill(*d, a, static_cast<hipStream_t>(stream)));
}

stepq_status stepq_linear_step(const stepq_linear_desc* d, int32_t batch, const int32_t* slot_ids,
                               int32_t num_slots, const void* q, int64_t q_stride, const void* k,
                               int64_t k_stride, const void* v, int64_t v_stride, const float* beta,
                               const float* gate, float* state, void* o, int64_t o_stride, void* stream) {
  stepq_status st = check_desc(d);
  if (st != STEPQ_OK) return st;
  if (batch < 0 || num_slots < 1) return STEPQ_ERR_INVALID_ARG;
  if (batch == 0) return STEPQ_OK;
  if (!slot_ids || !aligned(slot_ids, 4)) return STEPQ_ERR_INVALID_ARG;
  if (static_cast<int64_t>(batch) * d->num_heads > kMostHeads) return STEPQ_ERR_UNSUPPORTED;
  st = check_tensors(*d, q, q_stride, k, k_stride, v, v_stride, beta, gate, state, o, o_stride);
  if (st != STEPQ_OK) return st;
  stepq::LinearArgs a{};
  a.q = q; a.k = k; a.v = v;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.beta = beta; a.gate = gate;
  a.slot_ids = slot_ids;
  a.state = state; a.o = o; a.o_stride = o_stride;
  a.batch = batch; a.num_slots = num_slots;
  a.H = d->num_heads; a.rep = d->num_heads / d->num_qk_heads;
  return from_hip(stepq::launch_linear_step(*d, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
