// What beam_api.cpp hands to its launchers, with stand-ins for them: every row's tiles
// are covered by its parts for vocabularies up to the largest that is accepted, at
// every start of a row within 16 bytes.  Prints "ok <number of calls>".
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../../quantized_recurrent_state_packed_amd/csrc/beam_internal.hpp"

namespace {
stepq::SelectArgs seen;
}  // namespace

namespace stepq {
int select_parts(int64_t rows, int32_t vocab) {      // any split of up to 64 parts of a tile or more
  const int64_t tiles = (static_cast<int64_t>(vocab) + kTile - 1) / kTile, most = tiles < 64 ? tiles : 64;
  return static_cast<int>(rows < most ? most / rows : 1);
}
hipError_t launch_beam_select(const SelectArgs& a, int, hipStream_t) {
  seen = a;
  return hipSuccess;
}
hipError_t launch_beam_reorder(const ReorderArgs&, int32_t, uint32_t, hipStream_t) { return hipSuccess; }
}  // namespace stepq

int main() {
  int calls = 0;
  std::vector<int32_t> vocabs = {1, 1023, 1024, 1025, 65536, 131072};
  for (int32_t below = 0; below < 40; ++below) vocabs.push_back(0x7fffffff - stepq::kTile - below);
  void* const any = reinterpret_cast<void*>(4096);
  for (int32_t vocab : vocabs)
    for (int32_t beams : {1, 3, 64})
      for (int dtype : {STEPQ_F32, STEPQ_BF16, STEPQ_F16}) {
        const stepq_status s = stepq_beam_select(1, beams, vocab, 4, any, dtype, vocab, static_cast<float*>(any), nullptr, 0,
                                                 static_cast<int32_t*>(any), static_cast<int32_t*>(any),
                                                 static_cast<float*>(any), any, static_cast<size_t>(1) << 40, nullptr);
        if (s != STEPQ_OK) return std::printf("status %d for vocab %d\n", s, vocab), 1;
        const int64_t most = 16 / (dtype == STEPQ_F32 ? 4 : 2) - 1;     // elements before the row in its first 16 bytes
        if (seen.tiles < 1 || static_cast<int64_t>(seen.tiles) * seen.parts * stepq::kTile < vocab + most)
          return std::printf("vocab %d: %d parts of %d tiles\n", vocab, seen.parts, seen.tiles), 1;
        ++calls;
      }
  std::printf("ok %d\n", calls);
  return 0;
}
