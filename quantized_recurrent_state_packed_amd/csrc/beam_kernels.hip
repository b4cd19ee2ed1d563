// gfx950 kernels of beam search: selection over beams and vocabulary, and the
// reordering of state slots.
//
// Selection.  A beam's candidates are ordered by logit, which orders them by
// score too, so the best num_out of a beam need no softmax: one pass over the
// logits keeps a running maximum and sum of exponentials, and a list of the
// num_out largest.  A wave owns a stretch of a row (k_select_scan); its list is
// sorted across its lanes, one entry a lane.  k_select_merge joins a request's
// lists, turns logits into scores and orders the beams' candidates.
#include "beam_internal.hpp"

namespace stepq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kScanWaves = 4096;      // 256 compute units x 16 waves
constexpr int kPer = kTile / 64;      // logits a lane holds
constexpr float kInf = __builtin_inff();
constexpr float kLog2e = 1.4426950408889634f;

// List of a wave: entry i in lane i, best first; (-inf, -1) where there is
// none, which nothing ties with.
struct List {
  float x = -kInf;
  int32_t i = -1;
};

__device__ __forceinline__ bool better(float x, int32_t i, float y, int32_t j) { return x > y || (x == y && i < j); }

__device__ __forceinline__ float lane_value(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

// The value of the lane below (lane 0 keeps its own).
__device__ __forceinline__ int from_below(int x) {
  return __builtin_amdgcn_update_dpp(x, x, 0x138, 0xf, 0xf, false);   // wave_shr:1
}

// Inserts (x, i), the same in every lane, which beats the list's last entry.
__device__ __forceinline__ void insert(List& l, float x, int32_t i, int lane) {
  const bool after = better(x, i, l.x, l.i);
  const uint64_t m = __ballot(after);
  const float bx = __builtin_bit_cast(float, from_below(__builtin_bit_cast(int, l.x)));
  const int32_t bi = from_below(l.i);
  const bool here = lane == __builtin_ctzll(m | (1ull << 63));
  if (after) {
    l.x = here ? x : bx;
    l.i = here ? i : bi;
  }
}

// Offers every lane's (x, i), x >= floor, to the list, which keeps `n` entries that matter.
__device__ __forceinline__ void offer(List& l, float x, int32_t i, float floor, int n, int lane) {
  uint64_t m = __ballot(x >= floor && better(x, i, lane_value(l.x, n - 1), __builtin_amdgcn_readlane(l.i, n - 1)));
  while (m) {
    const int from = __builtin_ctzll(m);
    insert(l, lane_value(x, from), __builtin_amdgcn_readlane(i, from), lane);
    m &= m - 1;
    m &= __ballot(better(x, i, lane_value(l.x, n - 1), __builtin_amdgcn_readlane(l.i, n - 1)));
  }
}

// The n-th largest of the lanes' x, found bit by bit in the order of floats as
// integers.  Whatever is below it is not among the n largest of a set that x is part
// of: an empty list filled without it would take n (1 + ln(m / n)) insertions from m
// candidates, with it a few more than n.
__device__ __forceinline__ float nth_largest(float x, int n) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  const uint32_t key = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  uint32_t t = 0;
  for (uint32_t bit = 0x80000000u; bit; bit >>= 1)
    if (__popcll(__ballot(key >= (t | bit))) >= n) t |= bit;
  return __builtin_bit_cast(float, t ^ (t >> 31 ? 0x80000000u : 0xffffffffu));
}

// exp(x - m) for x <= m; 1 where both are the same infinity.
__device__ __forceinline__ float exp_below(float x, float m) {
  return x == m ? 1.0f : __builtin_amdgcn_exp2f((x - m) * kLog2e);
}

// kVec consecutive logits from a 16-byte boundary, as they lie in memory.
template <typename T>
struct Loader;
template <>
struct Loader<float> {
  static constexpr int kVec = 4;
  typedef f32x4 Raw;
  typedef float One;
  static constexpr One kNone = -kInf;
  static __device__ __forceinline__ float value(const Raw& r, int i) { return r[i]; }
};
template <>
struct Loader<__bf16> {
  static constexpr int kVec = 8;
  typedef u16x8 Raw;
  typedef uint16_t One;
  static constexpr One kNone = 0xff80;
  static __device__ __forceinline__ float value(const Raw& r, int i) {
    return __builtin_bit_cast(float, static_cast<uint32_t>(r[i]) << 16);
  }
};
template <>
struct Loader<_Float16> {
  static constexpr int kVec = 8;
  typedef u16x8 Raw;
  typedef uint16_t One;
  static constexpr One kNone = 0xfc00;
  static __device__ __forceinline__ float value(const Raw& r, int i) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(r[i])));
  }
};

// A tile of a row, -inf outside of it: a lane holds kVec neighbours from every 64 kVec.
template <typename T>
struct Tile {
  using L = Loader<T>;
  static constexpr int V = L::kVec;
  typename L::Raw raw[kPer / V];
  __device__ __forceinline__ void load(const T* row, int base, int vocab, int lane) {
    for (int e = 0; e < kPer / V; ++e) {
      const int at = base + (e * 64 + lane) * V;
      if (at >= 0 && at + V <= vocab) {
        raw[e] = *reinterpret_cast<const typename L::Raw*>(row + at);
      } else {
        for (int i = 0; i < V; ++i)
          raw[e][i] = at + i >= 0 && at + i < vocab ? reinterpret_cast<const typename L::One*>(row)[at + i] : L::kNone;
      }
    }
  }
};

// 32 x 8 rows of 131072 bfloat16 logits take 44 us, 1.5 TB/s; copying their bytes takes
// 13.  Bound by instructions, of the vector units first: counters say 21 of them and 15
// scalar ones a logit of every lane (insertions among them), the vector units busy 63 %
// of the time that a compute unit works, and 11 of its 16 waves under way on the average,
// which wait 41 % of their time, for loads and for the chain of their insertions.  With
// half as many waves 46.5 us, with twice as many 50 (every wave fills a list of its own).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_select_scan(SelectArgs p) {
  using L = Loader<T>;
  constexpr int V = L::kVec;
  const int lane = threadIdx.x & 63, n = p.num_out;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= static_cast<int64_t>(p.batch) * p.beams * p.parts) return;
  const int64_t row = unit / p.parts;
  const int part = static_cast<int>(unit % p.parts);
  const T* x = static_cast<const T*>(p.logits) + row * p.stride;
  // tiles begin at the 16-byte boundary at or below the row's start
  const int before = static_cast<int>((reinterpret_cast<uintptr_t>(x) % 16) / sizeof(T));
  const int tiles = static_cast<int>((static_cast<int64_t>(p.vocab) + before + kTile - 1) / kTile);
  const int begin = part * p.tiles, end = min(begin + p.tiles, tiles);
  List list;
  float m = -kInf, sum = 0.0f, last = -kInf;     // last: the list's n-th entry
  if (begin < end && (p.finished == nullptr || p.finished[row] == 0)) {
    Tile<T> next;
    next.load(x, begin * kTile - before, p.vocab, lane);
    for (int tile = begin; tile < end; ++tile) {
      const int base = tile * kTile - before;
      const Tile<T> now = next;
      if (tile + 1 < end) next.load(x, base + kTile, p.vocab, lane);
      float y[kPer];
      for (int e = 0; e < kPer; ++e) y[e] = L::value(now.raw[e / V], e % V);
      float top = fmaxf(y[0], -kInf);             // not NaN
      for (int e = 1; e < kPer; ++e) top = fmaxf(top, y[e]);
      const float most = fmaxf(m, top), from = most > -kInf ? most : 0.0f;
      float add = 0.0f;
      for (int e = 0; e < kPer; ++e) add += __builtin_amdgcn_exp2f((y[e] - from) * kLog2e);
      if (__ballot(!(add < kInf))) {              // a NaN, or an infinity, among the logits
        add = 0.0f;
        for (int e = 0; e < kPer; ++e) {
          y[e] = fmaxf(y[e], -kInf);
          add += y[e] > -kInf ? exp_below(y[e], most) : 0.0f;
        }
      }
      sum = (most > -kInf ? sum * exp_below(m, most) : 0.0f) + add;
      m = most;
      // tiles come in ascending order, so a tie with an entry of an earlier tile is lost
      if (__ballot(top > last)) {
        const float floor = tile == begin ? nth_largest(top, n) : last;
        for (int e = 0; e < kPer; ++e)
          if (__ballot(y[e] >= fmaxf(floor, last))) {
            offer(list, y[e], base + (e / V) * V * 64 + lane * V + e % V, floor, n, lane);
            last = lane_value(list.x, n - 1);
          }
      }
    }
    for (int s = 1; s < 64; s <<= 1) {
      const float om = __shfl_xor(m, s), os = __shfl_xor(sum, s);
      const float most = fmaxf(m, om);
      if (most > -kInf) sum = sum * exp_below(m, most) + os * exp_below(om, most);
      m = most;
    }
  }
  float* out = reinterpret_cast<float*>(p.workspace + unit * select_part_bytes(n));
  if (lane == 0) out[0] = m, out[1] = sum;
  if (lane < n) {
    out[2 + lane] = list.x;
    reinterpret_cast<int32_t*>(out)[2 + n + lane] = list.i;
  }
}

// A wave per beam joins the lists of the beam's parts, all of whose entries are
// loaded at once, and the first wave orders the beams' candidates.  Bound by the
// latency of its insertions: 17 us for 32 requests of 8 beams of 16 parts and 16
// candidates (waves wait 61 % of their time, 970 vector instructions each), 5.6 us for
// one of 4 beams of 32 parts and 4.
__global__ void __launch_bounds__(1024) k_select_merge(SelectArgs p) {
  __shared__ float sx[kMaxBeams][64];
  __shared__ int32_t si[kMaxBeams][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = p.num_out;
  const int64_t b = blockIdx.x;
  const size_t part_bytes = select_part_bytes(n);
  for (int beam = wave; beam < p.beams; beam += static_cast<int>(blockDim.x >> 6)) {
    const int64_t row = b * p.beams + beam;
    const float start = p.scores[row];
    float score = -kInf;
    int32_t token = -1;
    if (p.finished != nullptr && p.finished[row] != 0) {
      if (lane == 0) score = start, token = p.eos;
    } else {
      const uint8_t* in = p.workspace + row * p.parts * part_bytes;
      float m = -kInf, sum = 0.0f;
      if (lane < p.parts) {
        const float* head = reinterpret_cast<const float*>(in + lane * part_bytes);
        m = head[0], sum = head[1];
      }
      List list;
      constexpr int kAhead = 4;       // entries a lane loads at a time
      for (int first = 0; first < p.parts * n; first += 64 * kAhead) {
        float x[kAhead];
        int32_t i[kAhead];
        for (int a = 0; a < kAhead; ++a) {
          const int at = first + a * 64 + lane, part = at / n;
          const float* entry = reinterpret_cast<const float*>(in + min(part, p.parts - 1) * part_bytes) + 2 + at % n;
          x[a] = part < p.parts ? entry[0] : -kInf;
          i[a] = part < p.parts ? reinterpret_cast<const int32_t*>(entry)[n] : -1;
        }
        float floor = -kInf;
        if (first == 0) {
          float top = x[0];
          for (int a = 1; a < kAhead; ++a) top = fmaxf(top, x[a]);
          floor = nth_largest(top, n);
        }
        for (int a = 0; a < kAhead; ++a) offer(list, x[a], i[a], floor, n, lane);
      }
      for (int s = 1; s < 64; s <<= 1) {
        const float om = __shfl_xor(m, s), os = __shfl_xor(sum, s);
        const float now = fmaxf(m, om);
        if (now > -kInf) sum = sum * exp_below(m, now) + os * exp_below(om, now);
        m = now;
      }
      m = lane_value(m, 0), sum = lane_value(sum, 0);     // the lanes added in different orders
      if (list.x > -kInf) {
        score = start + ((list.x == m ? 0.0f : list.x - m) - logf(sum));
        token = list.i;
      }
    }
    sx[beam][lane] = lane < n && score > -kInf ? score : -kInf;   // a NaN score is none
    si[beam][lane] = token;
  }
  __syncthreads();
  if (wave != 0) return;
  List best;      // by score, then by place beam * 64 + rank
  float top = -kInf;
  for (int beam = 0; beam < p.beams; ++beam) top = fmaxf(top, sx[beam][lane]);
  const float floor = nth_largest(top, n);
  for (int beam = 0; beam < p.beams; ++beam) offer(best, sx[beam][lane], beam * 64 + lane, floor, n, lane);
  if (lane < n) {
    const bool some = best.x > -kInf;
    p.tokens[b * n + lane] = some ? si[best.i >> 6][best.i & 63] : -1;
    p.parents[b * n + lane] = some ? best.i >> 6 : -1;
    p.out_scores[b * n + lane] = best.x;
  }
}

// One workgroup per (new beam, segment of a slot).  Every wave works out the
// request's assignment from its parents: bit j of `first` says that new beam j
// is its parent's first child, bit i of `dead` that old beam i has none.  Only the
// states of beams that split are moved, each read and written once: 192 slots of
// 614 KB take 48.7 us, 4.85 TB/s, of the 45.7 that a copy takes.
__global__ void __launch_bounds__(kThreads) k_beam_reorder(ReorderArgs p) {
  const int lane = threadIdx.x & 63;
  const int j = blockIdx.x % p.beams;
  const int64_t base = static_cast<int64_t>(blockIdx.x) - j;
  const int32_t parent = lane < p.beams ? p.parents[base + lane] : -1;
  const uint64_t all = p.beams == 64 ? ~0ull : (1ull << p.beams) - 1;
  uint64_t first = 0, dead = 0;
  for (int i = 0; i < p.beams; ++i) {
    const uint64_t m = __ballot(parent == i);
    if (m) first |= m & (~m + 1);
    else dead |= 1ull << i;
  }
  const int32_t mine = __builtin_amdgcn_readlane(parent, j);
  const int32_t from = mine >= 0 && mine < p.beams ? p.slot_ids[base + mine] : -1;
  if (first >> j & 1) {
    if (blockIdx.y == 0 && threadIdx.x == 0) p.new_slot_ids[base + j] = from;
    return;
  }
  const int rank = __popcll(all & ~first & ((1ull << j) - 1));
  const bool pick = (dead >> lane & 1) && __popcll(dead & ((1ull << lane) - 1)) == rank;
  const int32_t to = p.slot_ids[base + __builtin_ctzll(__ballot(pick))];
  if (blockIdx.y == 0 && threadIdx.x == 0) p.new_slot_ids[base + j] = to;
  if (mine < 0 || mine >= p.beams || from < 0 || from >= p.num_slots || to < 0 || to >= p.num_slots) return;
  if (p.num_regions == 0) return;
  int r = 0;
  for (int lo = 1, hi = p.num_regions - 1; lo <= hi;) {
    const int mid = (lo + hi) / 2;
    if (p.regions[mid].first_segment <= blockIdx.y) r = mid, lo = mid + 1;
    else hi = mid - 1;
  }
  const uint64_t bytes = p.regions[r].slot_bytes;
  const uint64_t begin = static_cast<uint64_t>(blockIdx.y - p.regions[r].first_segment) * kSegment;
  const uint64_t end = begin + kSegment < bytes ? begin + kSegment : bytes;
  const uint8_t* src = p.regions[r].base + from * bytes;
  uint8_t* dst = p.regions[r].base + to * bytes;
  for (uint64_t at = begin + threadIdx.x * 16; at < end; at += kThreads * 16)
    *reinterpret_cast<u32x4*>(dst + at) = *reinterpret_cast<const u32x4*>(src + at);
}

}  // namespace

int select_parts(int64_t rows, int32_t vocab) {
  const int64_t tiles = (static_cast<int64_t>(vocab) + kTile - 1) / kTile;
  int64_t parts = rows > 0 ? (kScanWaves + rows - 1) / rows : 1;
  if (parts > 64) parts = 64;
  if (parts > tiles) parts = tiles;
  return static_cast<int>(parts);
}

hipError_t launch_beam_select(const SelectArgs& a, int dtype, hipStream_t s) {
  const int64_t units = static_cast<int64_t>(a.batch) * a.beams * a.parts;
  const dim3 grid(static_cast<uint32_t>((units + kWaves - 1) / kWaves));
  switch (dtype) {
    case STEPQ_BF16: k_select_scan<__bf16><<<grid, kThreads, 0, s>>>(a); break;
    case STEPQ_F16: k_select_scan<_Float16><<<grid, kThreads, 0, s>>>(a); break;
    default: k_select_scan<float><<<grid, kThreads, 0, s>>>(a); break;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int waves = a.beams < 16 ? a.beams : 16;
  k_select_merge<<<dim3(static_cast<uint32_t>(a.batch)), 64 * waves, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_beam_reorder(const ReorderArgs& a, int32_t batch, uint32_t segments, hipStream_t s) {
  k_beam_reorder<<<dim3(static_cast<uint32_t>(batch * a.beams), segments), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace stepq
