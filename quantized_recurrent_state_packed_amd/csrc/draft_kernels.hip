// gfx950 kernels of the verification of drafted tokens.
//
// k_verify_scan reads every row once and leaves the sums of its softmax, k_verify_pick decides
// how many drafts a request keeps, sums what the next token is drawn from over tiles of the one
// row that matters, and its last workgroup finds the token in the tile where the sum crosses the
// random number.
//
// A drawn token is a whole number that a difference in the last places of a sum can change:
// with sums good to d, one in 1 / (2 d tokens) draws near a border goes the other way, 3 % at
// 1e-7 over 131072 even tokens.  So exponentials and sums are binary64, whose multiplications
// run at the rate of binary32 ones here.
#include "draft_internal.hpp"

namespace stepq {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kPer = kVerifyTile / 64;      // logits a lane holds
constexpr float kInf = __builtin_inff();

template <typename T>
constexpr int kVec = 16 / sizeof(T);

// Consecutive logits, 16 bytes from any boundary of an element.
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Piece {
  T v[kVec<T>];
};

// A tile of a row in order of tokens, -inf outside of it: a lane holds kVec neighbours from
// every 64 kVec.
template <typename T>
struct Tile {
  static constexpr int V = kVec<T>;
  Piece<T> raw[kPer / V];
  static __device__ __forceinline__ int place(int e, int lane) { return (e / V * 64 + lane) * V + e % V; }
  __device__ __forceinline__ void load(const T* row, int base, int vocab, int lane) {
    for (int e = 0; e < kPer / V; ++e) {
      const int at = base + (e * 64 + lane) * V;
      if (at + V <= vocab) {
        raw[e] = *reinterpret_cast<const Piece<T>*>(row + at);
      } else {
        for (int i = 0; i < V; ++i) raw[e].v[i] = at + i < vocab ? row[at + i] : static_cast<T>(-kInf);
      }
    }
  }
  __device__ __forceinline__ float value(int e) const { return static_cast<float>(raw[e / V].v[e % V]); }
};

// 2^t good to 2e-15 of itself: the series of 2^f up to f^11, |f| <= 1/2.  Below 2^-1100, and for a
// NaN, 0.
__device__ __forceinline__ double power(double t) {
  t = fmax(t, -1100.0);
  const double n = rint(t), f = t - n;
  double s = 4.4455382718708114976e-10;                        // log(2)^k / k!
  s = fma(s, f, 7.0549116208011233299e-09);
  s = fma(s, f, 1.0178086009239699728e-07);
  s = fma(s, f, 1.3215486790144309488e-06);
  s = fma(s, f, 1.5252733804059840280e-05);
  s = fma(s, f, 1.5403530393381609954e-04);
  s = fma(s, f, 1.3333558146428443423e-03);
  s = fma(s, f, 9.6181291076284771619e-03);
  s = fma(s, f, 5.5504108664821579953e-02);
  s = fma(s, f, 2.4022650695910071233e-01);
  s = fma(s, f, 6.9314718055994530942e-01);
  s = fma(s, f, 1.0);
  return __builtin_amdgcn_ldexp(s, static_cast<int>(n));
}

// exp((x - m) / temperature) with c = log2(e) / temperature; an infinity shares with infinities alone.
__device__ __forceinline__ double weight(float x, float m, double c) {
  if (m == kInf) return x == kInf ? 1.0 : 0.0;
  return power((static_cast<double>(x) - static_cast<double>(m)) * c);
}

struct Request {
  int count;       // its drafts
  double c;        // log2(e) / temperature
  bool greedy;
};
__device__ __forceinline__ Request request_of(const VerifyArgs& p, int b) {
  Request r;
  r.count = p.num_drafts == nullptr ? p.drafts : max(0, min(p.drafts, p.num_drafts[b]));
  const float t = p.temperature == nullptr ? 1.0f : p.temperature[b];
  r.greedy = !(t > 0.0f);
  r.c = r.greedy ? 0.0 : 1.4426950408889634074 / static_cast<double>(t);
  return r;
}

__device__ __forceinline__ double across(double x, int s) {
  return __longlong_as_double(__shfl_xor(__double_as_longlong(x), s));
}

// A wave reads a part of a row.  Row r of a request is the target's of place r for r <= drafts,
// the draft's of place r - drafts - 1 beyond; rows behind the request's drafts are left out.
// Every lane keeps a reference m and its sum relative to it; m moves only when logits exceed it by
// a factor of 2^300, which binary64 holds, so sums are hardly ever rescaled.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_verify_scan(VerifyArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rows = 2 * p.drafts + 1;
  if (unit >= static_cast<int64_t>(p.batch) * rows * p.num_parts) return;
  const int part = static_cast<int>(unit % p.num_parts), r = static_cast<int>(unit / p.num_parts % rows);
  const int b = static_cast<int>(unit / p.num_parts / rows);
  if (part == 0 && r == 0 && lane == 0) p.arrived[b] = 0;
  const Request q = request_of(p, b);
  const bool drafted = r > p.drafts;
  const int place = drafted ? r - p.drafts - 1 : r;
  if (drafted ? place >= q.count || q.greedy || p.draft_logits == nullptr : place > q.count) return;
  const T* x = drafted ? static_cast<const T*>(p.draft_logits) + (static_cast<int64_t>(b) * p.drafts + place) * p.draft_stride
                       : static_cast<const T*>(p.logits) + (static_cast<int64_t>(b) * (p.drafts + 1) + place) * p.logits_stride;
  const int begin = min(part * p.part_tiles, p.tiles), end = min(begin + p.part_tiles, p.tiles);
  float m = -kInf;
  double sum = 0.0;
  int32_t at = -1;
  if (begin < end) {
    Tile<T> next;
    next.load(x, begin * kVerifyTile, p.vocab, lane);
    const float slack = static_cast<float>(fmin(300.0 / q.c, 1e30));
    for (int tile = begin; tile < end; ++tile) {
      const Tile<T> now = next;
      if (tile + 1 < end) next.load(x, (tile + 1) * kVerifyTile, p.vocab, lane);
      if (q.greedy) {
        for (int e = 0; e < kPer; ++e) {
          const float y = now.value(e);
          if (y > m) m = y, at = tile * kVerifyTile + Tile<T>::place(e, lane);      // ascending within a lane
        }
        continue;
      }
      float top = -kInf;
      for (int e = 0; e < kPer; ++e) top = fmaxf(top, now.value(e));               // not NaN
      if (__ballot(top > m + slack || (m == -kInf && top > m))) {
        if (top > m + slack || m == -kInf) {
          sum = m == -kInf || top == kInf ? 0.0 : sum * power((static_cast<double>(m) - static_cast<double>(top)) * q.c);
          m = top;
        }
      }
      if (__ballot(m == kInf)) {
        for (int e = 0; e < kPer; ++e) sum += m > -kInf ? weight(now.value(e), m, q.c) : 0.0;
      } else {
        const double from = m > -kInf ? m : 0.0;        // a lane without a logit that counts adds zeros
        double add = 0.0;
        for (int e = 0; e < kPer; ++e) add += power((static_cast<double>(now.value(e)) - from) * q.c);
        sum += add;
      }
    }
    if (q.greedy) {
      for (int s = 1; s < 64; s <<= 1) {
        const float om = __shfl_xor(m, s);
        const int32_t oa = __shfl_xor(at, s);
        if (om > m || (om == m && static_cast<uint32_t>(oa) < static_cast<uint32_t>(at))) m = om, at = oa;
      }
    } else {
      float most = m;
      for (int s = 1; s < 64; s <<= 1) most = fmaxf(most, __shfl_xor(most, s));
      sum = m == -kInf ? 0.0 : most == kInf ? (m == kInf ? sum : 0.0) : sum * power((static_cast<double>(m) - static_cast<double>(most)) * q.c);
      for (int s = 1; s < 64; s <<= 1) sum += across(sum, s);
      m = most;
    }
  }
  if (lane == 0) p.parts[unit] = {sum, m, at};
}

// A row's softmax: probabilities are weight(x, m, c) * scale.
struct Row {
  float m;
  int32_t at;
  double scale;      // 0: everything is banned
};

// The parts of a row, one a lane, joined; the same in every lane.
__device__ __forceinline__ Row join(const VerifyArgs& p, int64_t row, const Request& q, int lane) {
  VerifyPart v = {0.0, -kInf, -1};
  if (lane < p.num_parts) v = p.parts[row * p.num_parts + lane];
  Row r;
  r.m = v.m, r.at = v.at;
  for (int s = 1; s < 64; s <<= 1) {
    const float om = __shfl_xor(r.m, s);
    const int32_t oa = __shfl_xor(r.at, s);
    if (om > r.m || (om == r.m && static_cast<uint32_t>(oa) < static_cast<uint32_t>(r.at))) r.m = om, r.at = oa;
  }
  double sum = v.m == -kInf ? 0.0 : v.sum * (q.greedy ? 1.0 : weight(v.m, r.m, q.c));
  for (int s = 1; s < 64; s <<= 1) sum += across(sum, s);
  r.scale = sum > 0.0 ? 1.0 / sum : 0.0;
  return r;
}

// What the next token is drawn from.
struct Source {
  Row p, q;
  bool minus;         // p - q
  int32_t sharp;      // q is 1 at this token and nowhere else; -1: it is not
};

template <typename T>
__device__ __forceinline__ void shares(const Source& s, const T* x, const T* z, const Request& q, int tile, int vocab, int lane,
                                       double (&rest)[kPer], double (&whole)[kPer]) {
  Tile<T> a, d;
  a.load(x, tile * kVerifyTile, vocab, lane);
  const bool two = s.minus && s.sharp < 0;
  if (two) d.load(z, tile * kVerifyTile, vocab, lane);
  for (int e = 0; e < kPer; ++e) {
    whole[e] = s.p.scale > 0.0 ? weight(a.value(e), s.p.m, q.c) * s.p.scale : 0.0;
    rest[e] = whole[e];
    if (two && s.q.scale > 0.0) rest[e] = fmax(whole[e] - weight(d.value(e), s.q.m, q.c) * s.q.scale, 0.0);
    if (s.minus && s.sharp == tile * kVerifyTile + Tile<T>::place(e, lane)) rest[e] = 0.0;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_verify_pick(VerifyArgs p) {
  __shared__ Row joined[2 * kMostDrafts + 1];
  __shared__ double scan[kThreads];
  __shared__ int found[4];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x / p.pick_groups, g = blockIdx.x % p.pick_groups;
  const Request q = request_of(p, b);
  const int64_t row0 = static_cast<int64_t>(b) * (2 * p.drafts + 1);
  const bool sharp = q.greedy || p.draft_logits == nullptr;
  for (int r = w; r <= 2 * p.drafts; r += kWaves) {
    const int place = r > p.drafts ? r - p.drafts - 1 : r;
    if (r > p.drafts ? place >= q.count || sharp : place > q.count) continue;
    const Row j = join(p, row0 + r, q, lane);
    if (lane == 0) joined[r] = j;
  }
  __syncthreads();
  const T* target = static_cast<const T*>(p.logits) + static_cast<int64_t>(b) * (p.drafts + 1) * p.logits_stride;
  const T* draft = static_cast<const T*>(p.draft_logits) + static_cast<int64_t>(b) * p.drafts * p.draft_stride;
  // lane k looks at draft k
  bool good = false, known = false;
  int32_t token = -1;
  if (lane < q.count) {
    token = p.draft_tokens[b * static_cast<int64_t>(p.drafts) + lane];
    known = token >= 0 && token < p.vocab;
    if (known) {
      const Row t = joined[lane];
      if (q.greedy) {
        good = t.at == token;
      } else {
        const double pd = t.scale > 0.0 ? weight(static_cast<float>(target[lane * p.logits_stride + token]), t.m, q.c) * t.scale : 0.0;
        double qd = 1.0;
        if (!sharp) {
          const Row d = joined[p.drafts + 1 + lane];
          qd = d.scale > 0.0 ? weight(static_cast<float>(draft[lane * p.draft_stride + token]), d.m, q.c) * d.scale : 0.0;
        }
        good = static_cast<double>(p.uniforms[static_cast<int64_t>(b) * (p.drafts + 1) + lane]) * qd < pd;
      }
    }
  }
  const int n = __builtin_ctzll(~__ballot(good));          // at most 63 lanes are good
  const bool rejected = n < q.count && (__ballot(known) >> n & 1);
  int32_t* out = p.tokens + static_cast<int64_t>(b) * (p.drafts + 1);
  if (g == 0 && w == 0) {
    if (lane < n) out[lane] = token;
    if (lane > n && lane <= p.drafts) out[lane] = -1;
    if (lane == 0) p.accepted[b] = n;
    if (q.greedy && lane == 0) out[n] = joined[n].at;
  }
  if (q.greedy) return;
  Source s;
  s.p = joined[n];
  s.minus = rejected;
  s.sharp = sharp && rejected ? __shfl(token, n) : -1;
  if (s.minus && !sharp) s.q = joined[p.drafts + 1 + n];
  const T *x = target + n * p.logits_stride, *z = s.minus && !sharp ? draft + n * p.draft_stride : nullptr;
  double* sums = p.sums + static_cast<int64_t>(b) * p.tiles * 2;
  double rest[kPer], whole[kPer];
  for (int tile = g * kWaves + w; tile < p.tiles; tile += p.pick_groups * kWaves) {
    shares(s, x, z, q, tile, p.vocab, lane, rest, whole);
    double a = 0.0, c = 0.0;
    for (int e = 0; e < kPer; ++e) a += rest[e], c += whole[e];
    for (int k = 1; k < 64; k <<= 1) a += across(a, k), c += across(c, k);
    if (lane == 0) sums[2 * tile] = a, sums[2 * tile + 1] = c;
  }
  // the request's last workgroup goes on; nothing waits for it
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) found[0] = atomicAdd(p.arrived + b, 1u) == static_cast<uint32_t>(p.pick_groups) - 1;
  __syncthreads();
  if (!found[0]) return;
  __threadfence();
  // every thread takes a run of tiles; which sum counts depends on whether anything is left of p - q
  const int run = (p.tiles + kThreads - 1) / kThreads, from = min(static_cast<int>(threadIdx.x) * run, p.tiles);
  const int to = min(from + run, p.tiles);
  int which = 0;
  double total = 0.0;
  for (; which < 2; ++which) {
    double mine = 0.0;
    for (int tile = from; tile < to; ++tile) mine += sums[2 * tile + which];
    __syncthreads();
    scan[threadIdx.x] = mine;
    __syncthreads();
    total = 0.0;
    for (int k = 0; k < kThreads; ++k) {
      if (k == static_cast<int>(threadIdx.x)) mine = total;      // what lies before
      total += scan[k];
    }
    __syncthreads();
    scan[threadIdx.x] = mine;
    if (total > 0.0) break;
  }
  if (!(total > 0.0)) {
    if (threadIdx.x == 0) out[n] = -1;
    return;
  }
  const double goal = static_cast<double>(p.uniforms[static_cast<int64_t>(b) * (p.drafts + 1) + p.drafts]) * total;
  // the first tile whose sum crosses the goal, or the last that has any
  if (threadIdx.x == 0) found[1] = p.tiles, found[2] = -1;
  __syncthreads();
  double before = scan[threadIdx.x];
  for (int tile = from; tile < to; ++tile) {
    const double add = sums[2 * tile + which];
    if (add > 0.0) {
      atomicMax(&found[2], tile);
      if (before + add > goal) {
        atomicMin(&found[1], tile);
        break;
      }
    }
    before += add;
  }
  __syncthreads();
  const int tile = found[1] < p.tiles ? found[1] : found[2];
  if (tile >= from && tile < to) {
    double at = scan[threadIdx.x];
    for (int k = from; k < tile; ++k) at += sums[2 * k + which];
    scan[0] = at;             // one thread owns the tile, and the others are past their reads
  }
  __syncthreads();
  if (w != 0) return;
  double left = scan[0];
  shares(s, x, z, q, tile, p.vocab, lane, rest, whole);
  int32_t best = 0x7fffffff, last = -1;
  constexpr int V = kVec<T>;
  for (int e = 0; e < kPer; e += V) {
    double mine = 0.0;
    for (int i = 0; i < V; ++i) mine += which == 0 ? rest[e + i] : whole[e + i];
    double upto = mine;                                       // of the lanes up to this one
    for (int k = 1; k < 64; k <<= 1) {
      const double o = __longlong_as_double(__shfl_up(__double_as_longlong(upto), k));
      if (lane >= k) upto += o;
    }
    double at = left + (upto - mine);
    for (int i = 0; i < V; ++i) {
      const double v = which == 0 ? rest[e + i] : whole[e + i];
      at += v;
      const int32_t token_at = tile * kVerifyTile + Tile<T>::place(e + i, lane);
      if (v > 0.0) {
        last = max(last, token_at);
        if (at > goal) best = min(best, token_at);
      }
    }
    left += __longlong_as_double(__shfl(__double_as_longlong(upto), 63));
  }
  for (int k = 1; k < 64; k <<= 1) best = min(best, __shfl_xor(best, k)), last = max(last, __shfl_xor(last, k));
  if (lane == 0) out[n] = best != 0x7fffffff ? best : last;
}

template <typename T>
void launch(const VerifyArgs& a, hipStream_t s) {
  const int64_t units = static_cast<int64_t>(a.batch) * (2 * a.drafts + 1) * a.num_parts;
  k_verify_scan<T><<<dim3(static_cast<uint32_t>((units + kWaves - 1) / kWaves)), kThreads, 0, s>>>(a);
  if (hipPeekAtLastError() != hipSuccess) return;
  k_verify_pick<T><<<dim3(static_cast<uint32_t>(a.batch) * a.pick_groups), kThreads, 0, s>>>(a);
}

}  // namespace

hipError_t launch_verify(const VerifyArgs& a, int dtype, hipStream_t s) {
  if (dtype == STEPQ_BF16) launch<__bf16>(a, s);
  else if (dtype == STEPQ_F16) launch<_Float16>(a, s);
  else launch<float>(a, s);
  return hipGetLastError();
}

}  // namespace stepq
