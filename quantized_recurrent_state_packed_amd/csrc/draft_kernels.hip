// gfx950 kernels of the verification of drafted tokens.
//
// k_verify_scan reads every row once and leaves the sums of its softmax, k_verify_sums decides how many
// drafts a request keeps and sums what the next token is drawn from over tiles of the one row
// that matters, k_verify_choose finds the token in the tile where the sum crosses the random number.
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

// 2^t good to 3e-14 of itself: the polynomial that equals 2^f at the ten Chebyshev points of |f| <= 1/2.
// Below 2^-1100, and for a NaN, 0.
struct Power {
  double c[10] = {1.0000000000000144,    6.931471805599624e-01,  2.4022650695633263e-01, 5.550410866380432e-02,
                  9.618129195121405e-03, 1.33335583295702e-03,   1.5403433057773475e-04, 1.525259924712863e-05,
                  1.3259776859619875e-06, 1.0219919843734715e-07};
  // In scalar registers, which a multiplication takes as its addend; as constants the compiler would copy
  // five of them for every power.
  __device__ __forceinline__ Power() {
    for (int k = 0; k < 10; ++k) asm("" : "+s"(c[k]));
  }
  __device__ __forceinline__ double operator()(double t) const {
    t = fmax(t, -1100.0);
    const double n = rint(t), f = t - n;
    double s = fma(c[9], f, c[8]);
    for (int k = 7; k >= 0; --k) s = fma(s, f, c[k]);
    return __builtin_amdgcn_ldexp(s, static_cast<int>(n));
  }
};

// exp((x - m) / temperature) with c = log2(e) / temperature; an infinity shares with infinities alone.
__device__ __forceinline__ double weight(const Power& power, float x, float m, double c) {
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
// 64 requests of up to 5 drafts over 131072 bfloat16 logits take 61 us, 2.0 TB/s of the 123 MB of rows that are read: bound by vector
// instructions, 28 a logit, 17 of them binary64, units 81 % busy while a compute unit works, and by the last waves.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_verify_scan(VerifyArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rows = 2 * p.drafts + 1;
  if (unit >= static_cast<int64_t>(p.batch) * rows * p.num_parts) return;
  const int part = static_cast<int>(unit % p.num_parts), r = static_cast<int>(unit / p.num_parts % rows);
  const int b = static_cast<int>(unit / p.num_parts / rows);
  const Request q = request_of(p, b);
  const Power power;
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
        for (int e = 0; e < kPer; ++e) sum += m > -kInf ? weight(power, now.value(e), m, q.c) : 0.0;
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
      if (m == -kInf || (most == kInf && m < kInf)) sum = 0.0;
      else if (most < kInf) sum *= power((static_cast<double>(m) - static_cast<double>(most)) * q.c);
      for (int s = 1; s < 64; s <<= 1) sum += across(sum, s);
      m = most;
    }
  }
  if (lane == 0) p.parts[unit] = {sum, m, at};
}

// Joins the parts of a request's rows into LDS: `span` lanes (a power of two that holds num_parts) take a row.
__device__ __forceinline__ void join_rows(const VerifyArgs& p, const Power& power, int b, const Request& q, bool sharp,
                                          VerifyRow* joined) {
  const int span = p.num_parts <= 1 ? 1 : 1 << (32 - __builtin_clz(p.num_parts - 1));
  const int rows = 2 * p.drafts + 1, part = threadIdx.x & (span - 1);
  const int64_t row0 = static_cast<int64_t>(b) * rows;
  for (int first = 0; first < rows; first += kThreads / span) {
    const int r = first + static_cast<int>(threadIdx.x) / span, place = r > p.drafts ? r - p.drafts - 1 : r;
    const bool read = r < rows && (r > p.drafts ? place < q.count && !sharp : place <= q.count);
    VerifyPart v = {0.0, -kInf, -1};
    if (read && part < p.num_parts) v = p.parts[(row0 + r) * p.num_parts + part];
    float m = v.m;
    int32_t at = v.at;
    for (int s = 1; s < span; s <<= 1) {
      const float om = __shfl_xor(m, s);
      const int32_t oa = __shfl_xor(at, s);
      if (om > m || (om == m && static_cast<uint32_t>(oa) < static_cast<uint32_t>(at))) m = om, at = oa;
    }
    double sum = v.m == -kInf || q.greedy ? 0.0 : v.sum * weight(power, v.m, m, q.c);
    for (int s = 1; s < span; s <<= 1) sum += across(sum, s);
    if (read && part == 0) joined[r] = {sum > 0.0 ? 1.0 / sum : 0.0, m, at};
  }
  __syncthreads();
}

template <typename T>
__device__ __forceinline__ const T* target_row(const VerifyArgs& p, int b, int place) {
  return static_cast<const T*>(p.logits) + (static_cast<int64_t>(b) * (p.drafts + 1) + place) * p.logits_stride;
}
template <typename T>
__device__ __forceinline__ const T* draft_row(const VerifyArgs& p, int b, int place) {
  return static_cast<const T*>(p.draft_logits) + (static_cast<int64_t>(b) * p.drafts + place) * p.draft_stride;
}

// A tile of what the next token is drawn from, p - q, and of p alone.
template <typename T>
__device__ __forceinline__ void shares(const VerifyArgs& p, const Power& power, int b, const VerifyPlan& s, double c, int tile, int lane,
                                       double (&rest)[kPer], double (&whole)[kPer]) {
  const bool two = s.minus && s.sharp < 0 && s.q.scale > 0.0;
  Tile<T> a, d;
  a.load(target_row<T>(p, b, s.n), tile * kVerifyTile, p.vocab, lane);
  if (two) d.load(draft_row<T>(p, b, s.n), tile * kVerifyTile, p.vocab, lane);
  for (int e = 0; e < kPer; ++e) {
    whole[e] = s.p.scale > 0.0 ? weight(power, a.value(e), s.p.m, c) * s.p.scale : 0.0;
    rest[e] = whole[e];
  }
  if (two)
    for (int e = 0; e < kPer; ++e) rest[e] = fmax(whole[e] - weight(power, d.value(e), s.q.m, c) * s.q.scale, 0.0);
  if (s.minus && s.sharp >= 0)
    for (int e = 0; e < kPer; ++e)
      if (s.sharp == tile * kVerifyTile + Tile<T>::place(e, lane)) rest[e] = 0.0;
}

// 21 us for 64 requests of 131072 tokens: a row's two exponentials a token, and the chain of loads that decides the
// row (8 us for one request), which every workgroup of a request goes through for itself.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_verify_sums(VerifyArgs p) {
  __shared__ VerifyRow joined[2 * kMostDrafts + 1];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x / p.groups, g = blockIdx.x % p.groups;
  const Request q = request_of(p, b);
  const Power power;
  const bool sharp = q.greedy || p.draft_logits == nullptr;
  // lane k looks at draft k
  int32_t token = -1;
  float xt = 0.0f, zt = 0.0f, u = 0.0f;
  bool known = false;
  if (lane < q.count) {
    token = p.draft_tokens[b * static_cast<int64_t>(p.drafts) + lane];
    known = token >= 0 && token < p.vocab;
    u = p.uniforms[static_cast<int64_t>(b) * (p.drafts + 1) + lane];
    if (known && !q.greedy) {
      xt = static_cast<float>(target_row<T>(p, b, lane)[token]);
      if (!sharp) zt = static_cast<float>(draft_row<T>(p, b, lane)[token]);
    }
  }
  join_rows(p, power, b, q, sharp, joined);
  bool good = false;
  if (known) {
    const VerifyRow t = joined[lane];
    if (q.greedy) {
      good = t.at == token;
    } else {
      const double pd = t.scale > 0.0 ? weight(power, xt, t.m, q.c) * t.scale : 0.0;
      double qd = 1.0;
      if (!sharp) {
        const VerifyRow d = joined[p.drafts + 1 + lane];
        qd = d.scale > 0.0 ? weight(power, zt, d.m, q.c) * d.scale : 0.0;
      }
      good = static_cast<double>(u) * qd < pd;
    }
  }
  const int n = __builtin_ctzll(~__ballot(good));          // at most 63 lanes are good
  VerifyPlan s;
  s.n = n;
  s.p = joined[n];
  s.minus = n < q.count && (__ballot(known) >> n & 1);     // a draft was rejected
  s.sharp = s.minus && sharp ? __shfl(token, n) : -1;
  s.q = s.minus && !sharp ? joined[p.drafts + 1 + n] : VerifyRow{0.0, 0.0f, -1};
  s.pad = 0;
  if (g == 0 && w == 0) {
    int32_t* out = p.tokens + static_cast<int64_t>(b) * (p.drafts + 1);
    if (lane < n) out[lane] = token;
    if (lane > n && lane <= p.drafts) out[lane] = -1;
    if (lane == 0) {
      p.accepted[b] = n;
      p.plans[b] = s;
      if (q.greedy) out[n] = s.p.at;
    }
  }
  if (q.greedy) return;
  double* sums = p.sums + static_cast<int64_t>(b) * p.tiles * 2;
  double rest[kPer], whole[kPer];
  for (int tile = g * kWaves + w; tile < p.tiles; tile += p.groups * kWaves) {
    shares<T>(p, power, b, s, q.c, tile, lane, rest, whole);
    double a = 0.0, c = 0.0;
    for (int e = 0; e < kPer; ++e) a += rest[e], c += whole[e];
    // even lanes go on with one sum, odd lanes with the other
    double mine = lane & 1 ? c : a;
    mine += across(lane & 1 ? a : c, 1);
    for (int k = 2; k < 64; k <<= 1) mine += across(mine, k);
    if (lane < 2) sums[2 * tile + lane] = mine;
  }
}

// One workgroup a request: a chain of loads and sums across lanes, 7.6 us for 32 tiles, 12.4 for 64 requests of 128.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_verify_choose(VerifyArgs p) {
  __shared__ double waves[2][kWaves];
  __shared__ double start;
  __shared__ int found[2];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), b = blockIdx.x;
  const Request q = request_of(p, b);
  const Power power;
  if (q.greedy) return;
  const VerifyPlan s = p.plans[b];
  const float u = p.uniforms[static_cast<int64_t>(b) * (p.drafts + 1) + p.drafts];
  int32_t* out = p.tokens + static_cast<int64_t>(b) * (p.drafts + 1) + s.n;
  const double* sums = p.sums + static_cast<int64_t>(b) * p.tiles * 2;
  if (threadIdx.x == 0) found[0] = p.tiles, found[1] = -1;
  // every thread takes a run of tiles
  const int run = (p.tiles + kThreads - 1) / kThreads;
  const int from = min(static_cast<int>(threadIdx.x) * run, p.tiles), to = min(from + run, p.tiles);
  double mine[2] = {0.0, 0.0}, upto[2];
  for (int tile = from; tile < to; ++tile)
    for (int k = 0; k < 2; ++k) mine[k] += sums[2 * tile + k];
  for (int k = 0; k < 2; ++k) {
    upto[k] = mine[k];
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __longlong_as_double(__shfl_up(__double_as_longlong(upto[k]), d));
      if (lane >= d) upto[k] += o;
    }
    if (lane == 63) waves[k][w] = upto[k];
  }
  __syncthreads();
  double total[2], before[2];
  for (int k = 0; k < 2; ++k) {
    total[k] = 0.0;
    for (int v = 0; v < kWaves; ++v) {
      if (v == w) before[k] = total[k] + (upto[k] - mine[k]);
      total[k] += waves[k][v];
    }
  }
  const int which = total[0] > 0.0 ? 0 : 1;         // nothing is left of p - q: p
  if (!(total[which] > 0.0)) {
    if (threadIdx.x == 0) *out = -1;
    return;
  }
  const double goal = static_cast<double>(u) * total[which];
  // the first tile whose sum crosses the goal, or the last that has any
  double at = before[which];
  for (int tile = from; tile < to; ++tile) {
    const double add = sums[2 * tile + which];
    if (add > 0.0) {
      atomicMax(&found[1], tile);
      if (at + add > goal) {
        atomicMin(&found[0], tile);
        break;
      }
    }
    at += add;
  }
  __syncthreads();
  const int tile = found[0] < p.tiles ? found[0] : found[1];
  if (tile >= from && tile < to) {
    at = before[which];
    for (int k = from; k < tile; ++k) at += sums[2 * k + which];
    start = at;
  }
  __syncthreads();
  if (w != 0) return;
  double left = start;
  double rest[kPer], whole[kPer];
  shares<T>(p, power, b, s, q.c, tile, lane, rest, whole);
  int32_t best = 0x7fffffff, last = -1;
  constexpr int V = kVec<T>;
  for (int e = 0; e < kPer; e += V) {
    double own = 0.0;
    for (int i = 0; i < V; ++i) own += which == 0 ? rest[e + i] : whole[e + i];
    double all = own;                                         // of the lanes up to this one
    for (int k = 1; k < 64; k <<= 1) {
      const double o = __longlong_as_double(__shfl_up(__double_as_longlong(all), k));
      if (lane >= k) all += o;
    }
    double x = left + (all - own);
    for (int i = 0; i < V; ++i) {
      const double v = which == 0 ? rest[e + i] : whole[e + i];
      x += v;
      const int32_t token = tile * kVerifyTile + Tile<T>::place(e + i, lane);
      if (v > 0.0) {
        last = max(last, token);
        if (x > goal) best = min(best, token);
      }
    }
    left += __longlong_as_double(__shfl(__double_as_longlong(all), 63));
  }
  for (int k = 1; k < 64; k <<= 1) best = min(best, __shfl_xor(best, k)), last = max(last, __shfl_xor(last, k));
  if (lane == 0) *out = best != 0x7fffffff ? best : last;
}

template <typename T>
void launch(const VerifyArgs& a, hipStream_t s) {
  const int64_t units = static_cast<int64_t>(a.batch) * (2 * a.drafts + 1) * a.num_parts;
  k_verify_scan<T><<<dim3(static_cast<uint32_t>((units + kWaves - 1) / kWaves)), kThreads, 0, s>>>(a);
  if (hipPeekAtLastError() != hipSuccess) return;
  k_verify_sums<T><<<dim3(static_cast<uint32_t>(a.batch) * a.groups), kThreads, 0, s>>>(a);
  if (hipPeekAtLastError() != hipSuccess) return;
  k_verify_choose<T><<<dim3(static_cast<uint32_t>(a.batch)), kThreads, 0, s>>>(a);
}

}  // namespace

hipError_t launch_verify(const VerifyArgs& a, int dtype, hipStream_t s) {
  if (dtype == STEPQ_BF16) launch<__bf16>(a, s);
  else if (dtype == STEPQ_F16) launch<_Float16>(a, s);
  else launch<float>(a, s);
  return hipGetLastError();
}

}  // namespace stepq
