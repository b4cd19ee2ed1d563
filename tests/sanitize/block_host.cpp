// What scan_api.cpp, norm_api.cpp and draft_api.cpp hand to their launchers, with stand-ins for them: for random ragged
// requests every piece and every saved state has an index of its own below what the sizes allow, and every
// part of a workspace lies inside of it, apart from the others.  Prints "ok <number of calls>".
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>
#include <vector>

#include "../../quantized_recurrent_state_packed_amd/csrc/draft_internal.hpp"
#include "../../quantized_recurrent_state_packed_amd/csrc/norm_internal.hpp"
#include "../../quantized_recurrent_state_packed_amd/csrc/scan_internal.hpp"

namespace {
stepq::ScanArgs scan;
stepq::NormArgs norm;
stepq::VerifyArgs draft;
int calls = 0;

#define CHECK(x)                                              \
  do {                                                        \
    if (!(x)) {                                               \
      std::printf("line %d: %s\n", __LINE__, #x);             \
      std::exit(1);                                           \
    }                                                         \
  } while (0)
}  // namespace

namespace stepq {
hipError_t launch_scan_forward(const ScanArgs& a, int, hipStream_t) { return scan = a, ++calls, hipSuccess; }
hipError_t launch_scan_backward(const ScanArgs& a, int, hipStream_t) { return scan = a, ++calls, hipSuccess; }
hipError_t launch_scan_step(const ScanArgs& a, int, hipStream_t) { return scan = a, ++calls, hipSuccess; }
hipError_t launch_norm_forward(const NormArgs& a, int, hipStream_t) { return norm = a, ++calls, hipSuccess; }
hipError_t launch_norm_backward(const NormArgs& a, int, hipStream_t) { return norm = a, ++calls, hipSuccess; }
hipError_t launch_verify(const VerifyArgs& a, int, hipStream_t) { return draft = a, ++calls, hipSuccess; }
}  // namespace stepq

// Parts of a workspace, in order: each begins where the one before ends or later, and the last ends inside.
void in_order(std::vector<std::pair<const void*, size_t>> parts, const uint8_t* base, size_t bytes) {
  const uint8_t* at = base;
  for (const auto& p : parts) {
    if (p.first == nullptr) continue;
    const uint8_t* from = static_cast<const uint8_t*>(p.first);
    CHECK(from >= at && reinterpret_cast<uintptr_t>(from) % 16 == 0);
    at = from + p.second;
  }
  CHECK(at <= base + bytes);
}

void scans(std::mt19937& g) {
  uint8_t* const base = reinterpret_cast<uint8_t*>(1 << 20);
  void* const any = reinterpret_cast<void*>(4096);
  const std::vector<int> lengths = {0, 1, 7, 8, 9, 63, 64, 65, 127, 128, 129, 500, 20000};
  for (int round = 0; round < 300; ++round) {
    const int batch = 1 + static_cast<int>(g() % 9), width = 1 + static_cast<int>(g() % 300);
    std::vector<int64_t> cu = {static_cast<int64_t>(g() % 3)};
    for (int b = 0; b < batch; ++b) cu.push_back(cu.back() + lengths[g() % lengths.size()]);
    const int64_t total = cu.back() + g() % 5;
    const stepq_scan_desc d = {width, static_cast<int32_t>(g() % 3), 8.0f};
    const size_t bytes = stepq_scan_workspace_bytes(&d, batch, total), saved = stepq_scan_saved_bytes(&d, batch, total);
    float* f = static_cast<float*>(any);
    for (int back = 0; back < 2; ++back) {
      const int piece = stepq::scan_piece(d, total, batch, back == 1);
      const auto call = [&](size_t ws) {
        return back ? stepq_scan_backward(&d, batch, total, static_cast<int32_t*>(any), any, width, any, width, any, width, f, any, saved,
                                          any, width, nullptr, 0, nullptr, nullptr, any, width, any, width, any, width, f, base, ws, nullptr)
                    : stepq_scan_forward(&d, batch, total, static_cast<int32_t*>(any), any, width, any, width, any, width, f, nullptr, 0,
                                         nullptr, nullptr, any, width, any, saved, base, ws, nullptr);
      };
      CHECK(call(bytes) == STEPQ_OK && scan.piece == piece);
      const size_t n = static_cast<size_t>(scan.pieces) * width;
      const bool linked = scan.ticket != nullptr;
      int64_t longest = 0;
      for (int b = 0; b < batch; ++b) longest = std::max(longest, cu[b + 1] - cu[b]);
      CHECK(linked || longest <= piece);
      in_order({{scan.ticket, 16}, {scan.maps, n * 8}, {scan.ends, n * 8}, {scan.speeds, width * 4u}, {scan.partial, n * 4}}, base, bytes);
      if (linked) CHECK(static_cast<size_t>(scan.words) * 16 == static_cast<size_t>(reinterpret_cast<uint8_t*>(scan.speeds) - base));
      CHECK((scan.partial != nullptr) == (back == 1));
      std::set<int64_t> pieces, states;
      for (int b = 0; b < batch; ++b) {
        const int64_t count = cu[b + 1] - cu[b];
        for (int64_t tile = 0; tile == 0 || tile * piece < count; ++tile) {
          CHECK(pieces.insert(cu[b] / piece + b + tile).second && *pieces.rbegin() < scan.pieces);
        }
        for (int64_t t = 0; t < count; t += stepq::kBackTokens) {
          const int64_t at = cu[b] / stepq::kBackTokens + b + t / stepq::kBackTokens;
          CHECK(states.insert(at).second && (at + 1) * width * 4 <= static_cast<int64_t>(saved));
        }
      }
    }
  }
}

void norms() {
  uint8_t* const base = reinterpret_cast<uint8_t*>(1 << 20);
  void *a = reinterpret_cast<void*>(4096), *b = reinterpret_cast<void*>(8192), *c = reinterpret_cast<void*>(12288), *e = reinterpret_cast<void*>(16384);
  float* f = static_cast<float*>(a);
  for (int width : {1, 31, 32, 33, 128, 129, 512, 1024, 4096, 4097, 8192, 16384})
    for (int heads : {1, 3})
      for (int dtype : {STEPQ_F32, STEPQ_BF16})
        for (int64_t tokens : {1, 2, 700, 100000}) {
          const stepq_norm_desc d = {width, heads, dtype, STEPQ_GATE_SILU, 1, 1, 1e-6f};
          const int64_t row = static_cast<int64_t>(heads) * width;
          const size_t bytes = stepq_norm_workspace_bytes(&d, tokens);
          CHECK(stepq_norm_backward(&d, tokens, a, row, a, row, a, row, f, f, f, a, row, a, row, a, row, b, row, c, row, f, f, f, base,
                                    bytes, nullptr) == STEPQ_OK);
          CHECK(norm.groups >= 1 && static_cast<size_t>(norm.groups) * 3 * width * 4 <= bytes);
          CHECK(norm.heads == 1 && norm.block.stride == width && norm.rows == tokens * heads);
          CHECK(stepq_norm_backward(&d, tokens, a, row + 8, a, row, a, row, f, f, f, a, row, a, row, e, row, b, row, c, row, f, f, f, base,
                                    bytes, nullptr) == STEPQ_OK);
          CHECK(norm.heads == heads && norm.rows == tokens * heads);
          const stepq::NormShape s = stepq::norm_shape(width, dtype, true), t = stepq::norm_shape(width, dtype, false);
          const int vec = dtype == STEPQ_F32 ? 4 : 8;
          CHECK(s.lanes * s.pieces * vec >= width && t.lanes * t.pieces * vec >= width);
        }
}

void drafts() {
  uint8_t* const base = reinterpret_cast<uint8_t*>(1 << 20);
  void* const any = reinterpret_cast<void*>(4096);
  int32_t* i = static_cast<int32_t*>(any);
  for (int batch : {1, 2, 64, 5000})
    for (int k : {0, 1, 5, 63})
      for (int vocab : {1, 1023, 1024, 1025, 131072, 0x7fffffff - stepq::kVerifyTile}) {
        const size_t bytes = stepq_verify_workspace_bytes(batch, k, vocab);
        CHECK(bytes > 0);
        CHECK(stepq_verify_drafts(batch, k, vocab, any, STEPQ_BF16, vocab, any, vocab, i, nullptr, nullptr, static_cast<float*>(any), i,
                                  i, base, bytes, nullptr) == STEPQ_OK);
        const size_t rows = static_cast<size_t>(batch) * (2 * k + 1);
        CHECK(draft.num_parts >= 1 && draft.num_parts <= 64 && draft.groups >= 1);
        CHECK(static_cast<int64_t>(draft.tiles) * stepq::kVerifyTile >= vocab);
        CHECK(static_cast<int64_t>(draft.part_tiles) * draft.num_parts >= draft.tiles);
        in_order({{draft.parts, rows * draft.num_parts * sizeof(stepq::VerifyPart)}, {draft.plans, batch * sizeof(stepq::VerifyPlan)},
                  {draft.sums, static_cast<size_t>(batch) * draft.tiles * 16}}, base, bytes);
      }
}

int main() {
  std::mt19937 g(7);
  scans(g);
  norms();
  drafts();
  std::printf("ok %d\n", calls);
  return 0;
}
