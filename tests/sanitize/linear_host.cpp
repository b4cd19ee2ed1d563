// Which kernels prompts of 16-bit inputs reach, over descriptions, batches and lengths:
// linear_api.cpp with a stand-in for its launcher, which takes the launcher's decisions
// from the same rules.  Prints a line for every variant of the walk that is reached,
//   walk D parts delta tiles waves one-launch pass
// and of the chunk matrices, "chunks D parts delta"; fails where a call asks for a
// workspace that its own sizes exceed.
#include <cstdio>
#include <set>
#include <string>

#include "../../quantized_recurrent_state_packed_amd/csrc/linear_internal.hpp"

namespace {
std::set<std::string> reached;
void note(const char* format, int a, int b, int c, int d = 0, int e = 0, int f = 0, int g = 0) {
  char s[64];
  std::snprintf(s, sizeof s, format, a, b, c, d, e, f, g);
  reached.insert(s);
}
}  // namespace

namespace stepq {
hipError_t launch_linear_step(const stepq_linear_desc&, const LinearArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_linear_prefill(const stepq_linear_desc& d, const LinearArgs& a, hipStream_t) {
  if (d.dtype == STEPQ_F32) return hipSuccess;
  const int parts = d.dtype == STEPQ_BF16 ? 1 : 2, delta = d.rule == STEPQ_RULE_DELTA;
  const char* const walk = "walk %d %d %d %d %d %d %d";
  if (a.segment > 0) {
    note(walk, d.d, parts, delta, 1, d.d / 16, 1, 1);
    note(walk, d.d, parts, delta, 1, d.d / 16, 1, 2);
  } else if (a.apart) {
    note("chunks %d %d %d", d.d, parts, delta);
    note(walk, d.d, parts, delta, 1, apart_waves(d.d, parts, delta, static_cast<int64_t>(a.batch) * a.H), 0, 0);
  } else {
    note(walk, d.d, parts, delta, delta ? d.d / 64 : 1, delta ? 4 : d.d / 16, 1, 0);
  }
  return hipSuccess;
}
}  // namespace stepq

int main() {
  void* const any = reinterpret_cast<void*>(4096);
  const auto floats = static_cast<float*>(any);
  const auto ints = static_cast<int32_t*>(any);
  for (int d : {16, 32, 64, 128})
    for (int rule : {STEPQ_RULE_ADDITIVE, STEPQ_RULE_DELTA})
      for (int dtype : {STEPQ_F32, STEPQ_BF16, STEPQ_F16})
        for (int heads : {1, 8, 16, 48, 64, 100, 130, 300, 1000})
          for (int batch : {1, 2, 3, 5, 8, 16, 40})
            for (int64_t tokens : {0, 37, 64, 65, 700, 5000, 40000, 1000000}) {
              const stepq_linear_desc desc = {heads, heads, d, rule, dtype};
              const int64_t row = static_cast<int64_t>(heads) * d;
              const auto call = [&](void* workspace, size_t bytes) {
                return stepq_linear_prefill(&desc, batch, tokens, ints, any, row, any, row, any, row,
                                            rule == STEPQ_RULE_DELTA ? floats : nullptr, floats, ints, batch, nullptr, floats,
                                            any, row, workspace, bytes, nullptr);
              };
              const size_t bytes = stepq_linear_prefill_bytes(&desc, batch, tokens);
              const stepq_status s = call(bytes ? any : nullptr, bytes);
              if (bytes && (call(any, bytes - 1) != STEPQ_ERR_INVALID_ARG || call(nullptr, bytes) != STEPQ_ERR_INVALID_ARG))
                return std::printf("too little was accepted\n"), 1;
              for (int b = batch; b <= batch + 40; b += 13)        // a workspace for more is enough
                for (int64_t t : {tokens, tokens + 1, tokens + 64, tokens + 100000})
                  if (stepq_linear_workspace_bytes(&desc, b, t) < bytes) return std::printf("not enough for fewer\n"), 1;
              const bool one_launch = dtype != STEPQ_F32 && d >= 64 && batch * heads > 255;
              if (one_launch && bytes) return std::printf("one launch asks for %zu bytes\n", bytes), 1;
              const int32_t segment = stepq::segment_chunks(desc, tokens, batch);
              if (s != STEPQ_OK || (segment > 0 && static_cast<size_t>(stepq::max_segments(tokens, batch, segment)) * heads *
                                                           (d * d + stepq::kSegmentHead) * sizeof(float) > bytes))
                return std::printf("status %d, %zu bytes, d %d rule %d dtype %d heads %d batch %d tokens %lld\n", s, bytes, d,
                                   rule, dtype, heads, batch, static_cast<long long>(tokens)), 1;
            }
  for (const std::string& s : reached) std::printf("%s\n", s.c_str());
  return 0;
}
