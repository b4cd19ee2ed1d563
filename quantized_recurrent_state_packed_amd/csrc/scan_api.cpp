// Host side of the gated linear recurrence: argument checks, launches.  The
// operators are described in include/stepq_block.h.
#include "scan_internal.hpp"

#include <cmath>

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMostGroups = (1 << 23) - 1;   // workgroups of a call: a grid holds fewer than 2^32 threads

stepq_status check_desc(const stepq_scan_desc* d) {
  if (!d || d->width < 1) return STEPQ_ERR_INVALID_ARG;
  if (d->dtype != STEPQ_F32 && d->dtype != STEPQ_BF16 && d->dtype != STEPQ_F16) return STEPQ_ERR_INVALID_ARG;
  if (!std::isfinite(d->rate) || !(d->rate > 0.0f)) return STEPQ_ERR_INVALID_ARG;
  return d->width > (1 << 20) ? STEPQ_ERR_UNSUPPORTED : STEPQ_OK;
}

int elem_bytes(int dtype) { return dtype == STEPQ_F32 ? 4 : 2; }

// The sizes that the workspace functions and the calls over prompts share.
stepq_status check_sizes(const stepq_scan_desc* d, int32_t batch, int64_t total_tokens) {
  const stepq_status st = check_desc(d);
  if (st != STEPQ_OK) return st;
  if (batch < 0 || total_tokens < 0) return STEPQ_ERR_INVALID_ARG;
  if (total_tokens > 0x7fffffffLL) return STEPQ_ERR_UNSUPPORTED;
  const int64_t blocks = (d->width + 63) / 64;
  return stepq::scan_pieces(total_tokens, batch, stepq::kBackPiece) > kMostGroups / blocks ? STEPQ_ERR_UNSUPPORTED : STEPQ_OK;
}

// A tensor of tokens: [tokens][width], tokens `stride` apart.
bool rows_ok(const void* p, int64_t stride, const stepq_scan_desc& d) {
  return p && aligned(p, elem_bytes(d.dtype)) && stride >= d.width && stride <= (int64_t{1} << 24);
}

stepq_status check_slots(const int32_t* slot_ids, const float* state, int32_t num_slots) {
  if ((slot_ids != nullptr) != (state != nullptr)) return STEPQ_ERR_INVALID_ARG;
  if (slot_ids && (num_slots < 1 || !aligned(slot_ids, 4) || !aligned(state, 4))) return STEPQ_ERR_INVALID_ARG;
  return STEPQ_OK;
}

stepq_status from_hip(hipError_t e) { return e == hipSuccess ? STEPQ_OK : STEPQ_ERR_HIP; }

void place(stepq::ScanArgs& a, const stepq_scan_desc& d, void* workspace, const stepq::ScanWorkspace& w) {
  uint8_t* base = static_cast<uint8_t*>(workspace);
  if (w.maps > 0) {
    a.ticket = reinterpret_cast<uint32_t*>(base);
    a.maps = reinterpret_cast<uint64_t*>(base + w.maps);
    a.ends = reinterpret_cast<uint64_t*>(base + w.ends);
    a.speeds = reinterpret_cast<float*>(base + w.speeds);
    a.words = static_cast<int64_t>(w.speeds / 16);
  }
  if (w.bytes > w.partial) a.partial = reinterpret_cast<float*>(base + w.partial);
}

}  // namespace

extern "C" {

size_t stepq_scan_workspace_bytes(const stepq_scan_desc* d, int32_t batch, int64_t total_tokens) {
  if (check_sizes(d, batch, total_tokens) != STEPQ_OK) return 0;
  const size_t forward = stepq::scan_workspace(*d, total_tokens, batch, false).bytes;
  const size_t backward = stepq::scan_workspace(*d, total_tokens, batch, true).bytes;
  return forward > backward ? forward : backward;
}

size_t stepq_scan_saved_bytes(const stepq_scan_desc* d, int32_t batch, int64_t total_tokens) {
  if (check_sizes(d, batch, total_tokens) != STEPQ_OK) return 0;
  return stepq::scan_saved(*d, total_tokens, batch);
}

stepq_status stepq_scan_forward(const stepq_scan_desc* d, int32_t batch, int64_t total_tokens, const int32_t* cu_seqlens,
                                const void* x, int64_t x_stride, const void* gate_a, int64_t gate_a_stride,
                                const void* gate_x, int64_t gate_x_stride, const float* decay, const int32_t* slot_ids,
                                int32_t num_slots, const uint8_t* resume, float* state, void* y, int64_t y_stride,
                                void* saved, size_t saved_bytes, void* workspace, size_t workspace_bytes, void* stream) {
  stepq_status st = check_sizes(d, batch, total_tokens);
  if (st != STEPQ_OK) return st;
  if (batch == 0) return STEPQ_OK;
  if (!cu_seqlens || !aligned(cu_seqlens, 4) || !decay || !aligned(decay, 4)) return STEPQ_ERR_INVALID_ARG;
  if (!rows_ok(x, x_stride, *d) || !rows_ok(gate_a, gate_a_stride, *d) || !rows_ok(gate_x, gate_x_stride, *d) ||
      !rows_ok(y, y_stride, *d))
    return STEPQ_ERR_INVALID_ARG;
  st = check_slots(slot_ids, state, num_slots);
  if (st != STEPQ_OK) return st;
  if (saved && (!aligned(saved, 16) || saved_bytes < stepq_scan_saved_bytes(d, batch, total_tokens)))
    return STEPQ_ERR_INVALID_ARG;
  const stepq::ScanWorkspace w = stepq::scan_workspace(*d, total_tokens, batch, false);
  if (w.bytes > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < w.bytes)) return STEPQ_ERR_INVALID_ARG;
  stepq::ScanArgs a{};
  a.x = x; a.ga = gate_a; a.gx = gate_x; a.y = y;
  a.x_stride = x_stride; a.ga_stride = gate_a_stride; a.gx_stride = gate_x_stride; a.y_stride = y_stride;
  a.decay = decay; a.cu_seqlens = cu_seqlens; a.slot_ids = slot_ids; a.resume = resume; a.state = state;
  a.saved = static_cast<float*>(saved);
  a.total_tokens = total_tokens; a.batch = batch; a.num_slots = num_slots; a.width = d->width; a.rate = d->rate;
  a.piece = stepq::scan_piece(*d, total_tokens, batch, false);
  a.pieces = static_cast<uint32_t>(stepq::scan_pieces(total_tokens, batch, a.piece));
  place(a, *d, workspace, w);
  return from_hip(stepq::launch_scan_forward(a, d->dtype, static_cast<hipStream_t>(stream)));
}

stepq_status stepq_scan_backward(const stepq_scan_desc* d, int32_t batch, int64_t total_tokens, const int32_t* cu_seqlens,
                                 const void* x, int64_t x_stride, const void* gate_a, int64_t gate_a_stride,
                                 const void* gate_x, int64_t gate_x_stride, const float* decay, const void* saved,
                                 size_t saved_bytes, const void* dy, int64_t dy_stride, const int32_t* slot_ids,
                                 int32_t num_slots, const uint8_t* resume, float* dstate, void* dx, int64_t dx_stride,
                                 void* dgate_a, int64_t dgate_a_stride, void* dgate_x, int64_t dgate_x_stride, float* ddecay,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  stepq_status st = check_sizes(d, batch, total_tokens);
  if (st != STEPQ_OK) return st;
  if (!decay || !aligned(decay, 4) || !ddecay || !aligned(ddecay, 4)) return STEPQ_ERR_INVALID_ARG;
  const stepq::ScanWorkspace w = stepq::scan_workspace(*d, total_tokens, batch, true);
  if (batch > 0) {
    if (!cu_seqlens || !aligned(cu_seqlens, 4)) return STEPQ_ERR_INVALID_ARG;
    if (!rows_ok(x, x_stride, *d) || !rows_ok(gate_a, gate_a_stride, *d) || !rows_ok(gate_x, gate_x_stride, *d) ||
        !rows_ok(dy, dy_stride, *d) || !rows_ok(dx, dx_stride, *d) || !rows_ok(dgate_a, dgate_a_stride, *d) ||
        !rows_ok(dgate_x, dgate_x_stride, *d))
      return STEPQ_ERR_INVALID_ARG;
    st = check_slots(slot_ids, dstate, num_slots);
    if (st != STEPQ_OK) return st;
    if (!saved || !aligned(saved, 16) || saved_bytes < stepq_scan_saved_bytes(d, batch, total_tokens))
      return STEPQ_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < w.bytes) return STEPQ_ERR_INVALID_ARG;
  }
  stepq::ScanArgs a{};
  a.x = x; a.ga = gate_a; a.gx = gate_x; a.dy = dy; a.y = dx; a.dga = dgate_a; a.dgx = dgate_x;
  a.x_stride = x_stride; a.ga_stride = gate_a_stride; a.gx_stride = gate_x_stride; a.dy_stride = dy_stride;
  a.y_stride = dx_stride; a.dga_stride = dgate_a_stride; a.dgx_stride = dgate_x_stride;
  a.decay = decay; a.cu_seqlens = cu_seqlens; a.slot_ids = slot_ids; a.resume = resume; a.state = dstate;
  a.saved = const_cast<float*>(static_cast<const float*>(saved));
  a.ddecay = ddecay;
  a.total_tokens = total_tokens; a.batch = batch; a.num_slots = num_slots; a.width = d->width; a.rate = d->rate;
  a.piece = stepq::scan_piece(*d, total_tokens, batch, true);
  a.pieces = static_cast<uint32_t>(stepq::scan_pieces(total_tokens, batch, a.piece));
  if (batch == 0) a.pieces = 0;
  else place(a, *d, workspace, w);
  return from_hip(stepq::launch_scan_backward(a, d->dtype, static_cast<hipStream_t>(stream)));
}

stepq_status stepq_scan_step(const stepq_scan_desc* d, int32_t batch, const int32_t* slot_ids, int32_t num_slots,
                             const void* x, int64_t x_stride, const void* gate_a, int64_t gate_a_stride,
                             const void* gate_x, int64_t gate_x_stride, const float* decay, float* state, void* y,
                             int64_t y_stride, void* stream) {
  stepq_status st = check_desc(d);
  if (st != STEPQ_OK) return st;
  if (batch < 0 || num_slots < 1) return STEPQ_ERR_INVALID_ARG;
  if (batch == 0) return STEPQ_OK;
  if (batch > kMostGroups / ((d->width + 255) / 256)) return STEPQ_ERR_UNSUPPORTED;
  if (!slot_ids || !state || !decay || !aligned(decay, 4)) return STEPQ_ERR_INVALID_ARG;
  if (!rows_ok(x, x_stride, *d) || !rows_ok(gate_a, gate_a_stride, *d) || !rows_ok(gate_x, gate_x_stride, *d) ||
      !rows_ok(y, y_stride, *d))
    return STEPQ_ERR_INVALID_ARG;
  st = check_slots(slot_ids, state, num_slots);
  if (st != STEPQ_OK) return st;
  stepq::ScanArgs a{};
  a.x = x; a.ga = gate_a; a.gx = gate_x; a.y = y;
  a.x_stride = x_stride; a.ga_stride = gate_a_stride; a.gx_stride = gate_x_stride; a.y_stride = y_stride;
  a.decay = decay; a.slot_ids = slot_ids; a.state = state;
  a.batch = batch; a.num_slots = num_slots; a.width = d->width; a.rate = d->rate;
  return from_hip(stepq::launch_scan_step(a, d->dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
