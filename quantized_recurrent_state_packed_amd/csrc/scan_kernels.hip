// gfx950 kernels of the gated linear recurrence: ragged prompts, their backward
// pass, and single tokens.
//
//   a_t = exp(-rate s(ga_t) softplus(decay)),  b_t = sqrt(1 - a_t^2)
//   h_t = a_t h_{t-1} + u_t,  u_t = b_t s(gx_t) x_t,  y_t = h_t
//
// A run of tokens is an affine map of the state before it, h -> A h + B, and maps
// of neighbouring runs compose.  A wave holds some tokens of 64 V channels in registers,
// the waves of a workgroup follow each other in time and make up a piece.  Each wave works
// out its map, the maps meet in LDS, states are handed on from piece to piece (hand_on), and
// every wave walks its tokens from the state that it starts from.  So every tensor is read or
// written once, whatever a request's length, and one long request spreads over the chip
// like many short ones.
//
// Backward, with c_t = a_{t+1} g_{t+1} what comes from the tokens behind (the final
// state's gradient for the last one), g_t = dy_t + c_t:
//   dx_t = g_t b_t s(gx_t),   dgx_t = g_t u_t (1 - s(gx_t))
//   P_t = (d log a_t) log a_t = g_t (a_t h_{t-1} log a_t - a_t^2 s(gx_t) x_t log a_t / b_t)
//   dga_t = P_t (1 - s(ga_t)),   ddecay = sum_t P_t s(decay) / softplus(decay)
// c is a recurrence of the same kind, backwards: c -> a_t c + a_t dy_t.  log a / b goes to 0
// with log a, like -sqrt(-log a / 2).
#include <type_traits>

#include "scan_internal.hpp"

namespace stepq {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2 = 0.6931471805599453f;

// V neighbouring channels of a token, as they lie in memory until they are used: 16-bit pairs stay in
// one register.
template <int BYTES>
struct Word;
template <>
struct Word<2> { typedef uint16_t type; };
template <>
struct Word<4> { typedef uint32_t type; };

template <typename T, int V>
struct Vec {
  typedef typename Word<sizeof(T) * V>::type Raw;
  Raw raw;
  __device__ __forceinline__ float operator[](int v) const {
    if constexpr (sizeof(T) == 4) {
      return __builtin_bit_cast(float, raw);
    } else if constexpr (std::is_same<T, __bf16>::value) {
      if constexpr (V == 1) return __builtin_bit_cast(float, static_cast<uint32_t>(raw) << 16);
      else return __builtin_bit_cast(float, v ? raw & 0xffff0000u : raw << 16);
    } else {
      return static_cast<float>(__builtin_bit_cast(T, static_cast<uint16_t>(v ? static_cast<uint32_t>(raw) >> 16 : raw)));
    }
  }
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load(const T* p) {
  return {*reinterpret_cast<const typename Vec<T, V>::Raw*>(p)};
}
template <typename T, int V>
__device__ __forceinline__ typename Vec<T, V>::Raw rounded(const float (&x)[V]) {
  typedef T Some __attribute__((ext_vector_type(V)));
  Some r;
  for (int i = 0; i < V; ++i) r[i] = static_cast<T>(x[i]);
  return __builtin_bit_cast(typename Vec<T, V>::Raw, r);
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&x)[V]) {
  *reinterpret_cast<typename Vec<T, V>::Raw*>(p) = rounded<T, V>(x);
}

// Keeps the compiler from holding on to what it worked out of these values before.
template <typename T, int V>
__device__ __forceinline__ void again(Vec<T, V>& x) {
  if constexpr (sizeof(x) >= 4) asm volatile("" : "+v"(x.raw));
}

__device__ __forceinline__ float logistic(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// 1 - 2^z for z <= 0.  Up to |z| = 1/2 the polynomial of degree 4 that equals (1 - 2^z) / -z at the five Chebyshev
// points of that range, which is off by 1.4e-8 of it at most, 1.3e-7 with binary32's roundings (the series up to z^5
// up to 1/4 was off by 3.2e-7); beyond it the difference, off by a step of 2^z, 2e-7 of it at worst.  The retention, 1 less
// this, has half a step's error of its own either way.
__device__ __forceinline__ float one_less_exp2(float z) {
  float s = 1.15543997e-03f;
  s = fmaf(s, z, 9.54227503e-03f);
  s = fmaf(s, z, 5.54907198e-02f);
  s = fmaf(s, z, 2.40225675e-01f);
  s = fmaf(s, z, 6.93147172e-01f);
  const float far = 1.0f - __builtin_amdgcn_exp2f(z);
  return z > -0.5f ? -z * s : far;
}

// -rate softplus(decay) log2(e), the binary logarithm of the retention at an open gate; log1p by the
// quotient that takes the rounding of 1 + e back out.
__device__ __forceinline__ float speed_of(float decay, float rate) {
  const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(decay));
  const float w = 1.0f + e;
  const float l = w == 1.0f ? e : logf(w) * (e / (w - 1.0f));
  return -rate * kLog2e * (fmaxf(decay, 0.0f) + l);
}

// The request whose pieces hold index `piece`, and which of them it is.
struct Piece {
  int request;      // -1: none
  int64_t first;    // token index of the request's first row
  int32_t count;    // its tokens
  int32_t tile;     // which of its pieces
};

__device__ __forceinline__ int64_t start_of(const ScanArgs& p, int b) {
  const int64_t at = p.cu_seqlens[b];
  return at < 0 ? 0 : at > p.total_tokens ? p.total_tokens : at;
}

// The last request that begins at this index or before it, 64 at a time.
template <int PIECE>
__device__ __forceinline__ Piece find(const ScanArgs& p, int64_t piece) {
  const int lane = threadIdx.x & 63;
  Piece r = {-1, 0, 0, 0};
  int from = 0, n = p.batch;
  for (bool more = true; more;) {
    const int step = (n + 63) / 64, at = from + lane * step;
    const bool before = lane * step < n && start_of(p, at) / PIECE + at <= piece;
    const int count = __popcll(__ballot(before));
    if (count == 0) return r;                 // rows before the first request
    from += (count - 1) * step;
    n = min(step, n - (count - 1) * step);
    more = step > 1;
  }
  // the same in all lanes, and the compiler is to know: addresses of rows stay in scalar registers
  from = __builtin_amdgcn_readfirstlane(from);
  r.request = from;
  const int32_t first = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(start_of(p, from)));
  const int32_t end = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(start_of(p, from + 1)));
  r.first = first;
  r.count = end > first ? end - first : 0;
  r.tile = static_cast<int32_t>(piece - (r.first / PIECE + from));
  if (r.tile < 0 || (r.tile > 0 && static_cast<int64_t>(r.tile) * PIECE >= r.count)) r.request = -1;
  return r;
}

// Some tokens' rows: the first one's start in scalar registers, a lane's offset from there in 32 bits
// (strides are at most 2^24 elements).
template <typename T, int V>
struct Rows {
  typedef __attribute__((address_space(1))) typename Vec<T, V>::Raw Global;
  typedef __attribute__((address_space(1))) char Byte;
  uint64_t first;
  uint32_t stride, column;      // bytes
  __device__ __forceinline__ Rows(const void* p, int64_t stride, int64_t row, uint32_t column)
      : first(reinterpret_cast<uint64_t>(static_cast<const T*>(p) + row * stride)), stride(static_cast<uint32_t>(stride * sizeof(T))),
        column(static_cast<uint32_t>(column * sizeof(T))) {
    asm("" : "+s"(first));
  }
  __device__ __forceinline__ Global* at(int t) const {
    return reinterpret_cast<Global*>(reinterpret_cast<Byte*>(first) + (static_cast<uint32_t>(t) * stride + column));
  }
  __device__ __forceinline__ Vec<T, V> load(int t) const { return {*at(t)}; }
  __device__ __forceinline__ void store(int t, const float (&x)[V]) const { *at(t) = rounded<T, V>(x); }
};

__device__ __forceinline__ int slot_of(const ScanArgs& p, int b) {
  if (p.slot_ids == nullptr) return -1;
  const int slot = __builtin_amdgcn_readfirstlane(p.slot_ids[b]);
  return slot >= 0 && slot < p.num_slots ? slot : -2;     // -2: not a slot
}

// Handing states on between workgroups.  A workgroup takes the next piece in order by a ticket, so
// all that it waits for has been taken by workgroups that run already and that wait for none
// behind them: every wait ends.  (Every workgroup publishes its words, also for pieces that turn out
// to hold no tokens, so this does not depend on what cu_seqlens holds.)  A word is 8 bytes, written
// and read at once and all ones until then, so it needs no flag and no fence.
// A piece's map is published in `maps` as soon as its tokens are read.  W pieces make a group (W waves of
// a workgroup, one looking at each map), W groups a run: a group's last piece publishes the group's
// map in `ends` when it has the maps of the others, a run's last piece the state behind it, as a
// constant map.  A piece applies the state before its run, the maps of the groups before its own and
// those of the pieces before it.  So states go from run to run, W W pieces at a time, and what one workgroup waits for
// another is some microseconds in thousands of tokens.  How a state is put together depends on places alone, never
// on what came first.
constexpr uint64_t kNone = ~0ull;

__device__ __forceinline__ uint64_t pack(float a, float b) {
  if (a != a) a = __builtin_nanf("");          // no NaN reads as an empty word
  return static_cast<uint64_t>(__builtin_bit_cast(uint32_t, a)) << 32 | __builtin_bit_cast(uint32_t, b);
}
template <int V>
__device__ __forceinline__ void publish(uint64_t* words, int64_t index, int width, int c, const float (&a)[V],
                                        const float (&b)[V]) {
  if (c >= width) return;
  for (int v = 0; v < V; ++v)
    __hip_atomic_store(words + index * width + c + v, pack(a[v], b[v]), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <int V>
__device__ __forceinline__ void wait_for(const uint64_t* words, int64_t index, int width, int c, float (&a)[V], float (&b)[V]) {
  const uint64_t* at = words + index * width + (c < width ? c : 0);
  uint64_t word[V];
  for (int v = 0; v < V; ++v) word[v] = c < width ? kNone : 0;
  for (;;) {
    bool all = true;
    for (int v = 0; v < V; ++v) {
      if (word[v] == kNone) word[v] = __hip_atomic_load(at + v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      all = all && word[v] != kNone;
    }
    if (!__ballot(!all)) break;
    __builtin_amdgcn_s_sleep(1);
  }
  for (int v = 0; v < V; ++v) {
    a[v] = __builtin_bit_cast(float, static_cast<uint32_t>(word[v] >> 32));
    b[v] = __builtin_bit_cast(float, static_cast<uint32_t>(word[v]));
  }
}

// The request's state, before the barrier behind which its first piece publishes: whoever overwrites the
// slot has waited for that.
template <int V>
__device__ __forceinline__ void state_of(const ScanArgs& p, int slot, bool from, int c, float (&h)[V]) {
  for (int v = 0; v < V; ++v) {
    h[v] = from ? p.state[static_cast<int64_t>(slot) * p.width + c + v] : 0.0f;
    asm volatile("" : "+v"(h[v]));       // its value, not its load, is here
  }
}

// The workspace before the pieces run, and every channel's speed: 4 us for 17 MB of words (32768 tokens x 4096).
__global__ void __launch_bounds__(256) k_scan_clear(ScanArgs p) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4* to = reinterpret_cast<u32x4*>(p.ticket);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = i0; i < p.words; i += step) to[i] = u32x4{~0u, ~0u, ~0u, ~0u};
  for (int64_t c = i0; c < p.width; c += step) p.speeds[c] = speed_of(p.decay[c], p.rate);
}

// LDS of a workgroup's waves' maps, and of the maps before it: of pieces, of groups, and of runs.
template <int V, int W>
struct Shared {
  float own[W][2][64 * V];
  float pieces[W - 1][2][64 * V];
  float groups[W][2][64 * V];        // the last one: the state before the run
  uint32_t ticket;
};

template <int V>
__device__ __forceinline__ void write(float (&to)[2][64 * V], int lane, const float (&a)[V], const float (&b)[V]) {
  for (int v = 0; v < V; ++v) to[0][lane * V + v] = a[v], to[1][lane * V + v] = b[v];
}
template <int V>
__device__ __forceinline__ void apply(const float (&map)[2][64 * V], int lane, float (&h)[V]) {
  for (int v = 0; v < V; ++v) h[v] = fmaf(map[0][lane * V + v], h[v], map[1][lane * V + v]);
}

// (a, b) becomes the map of what it was of and then of this one.
template <int V>
__device__ __forceinline__ void compose(const float (&map)[2][64 * V], int lane, float (&a)[V], float (&b)[V]) {
  for (int v = 0; v < V; ++v) {
    const float m = map[0][lane * V + v];
    a[v] *= m, b[v] = fmaf(m, b[v], map[1][lane * V + v]);
  }
}

// From the waves' maps, in order of time w = 0 .. W - 1, the state that each wave starts from, and the one
// behind the last.  `index`: of this piece; `ahead`: +1 where pieces follow each other by rising index, -1 where
// by falling; `place`: this piece's among its request's, from the end that the states come
// from; h: the request's state there, used by its first piece.
template <int V, int W, bool LINKED>
__device__ __forceinline__ void hand_on(const ScanArgs& p, Shared<V, W>& s, int w, int lane, int64_t index, int ahead, int place,
                                        int c, const float (&A)[V], const float (&B)[V], float (&h)[V], float (&end)[V]) {
  write<V>(s.own[w], lane, A, B);
  __syncthreads();
  // pieces of its group, groups of its run before this one; where the run begins
  const int behind = LINKED ? place % W : 0, groups = LINKED ? place / W % W : 0, run = LINKED ? place % (W * W) : 0;
  if (LINKED) {
    float a[V], b[V];
    if (w == W - 1) {
      for (int v = 0; v < V; ++v) a[v] = 1.0f, b[v] = 0.0f;
      for (int k = 0; k < W; ++k) compose<V>(s.own[k], lane, a, b);
      if (place == 0)          // the request's first piece knows its state: its map is a constant
        for (int v = 0; v < V; ++v) b[v] = fmaf(a[v], h[v], b[v]), a[v] = 0.0f;
      publish<V>(p.maps, index, p.width, c, a, b);
      if (behind != W - 1) publish<V>(p.ends, index, p.width, c, a, b);       // nobody asks for it
    } else if (w < behind) {
      wait_for<V>(p.maps, index - static_cast<int64_t>(ahead) * (behind - w), p.width, c, a, b);
      write<V>(s.pieces[w], lane, a, b);
    }
    __syncthreads();
    if (w == W - 1 && behind == W - 1 && run != W * W - 1) {
      float ga[V], gb[V];
      for (int v = 0; v < V; ++v) ga[v] = 1.0f, gb[v] = 0.0f;
      for (int k = 0; k < W - 1; ++k) compose<V>(s.pieces[k], lane, ga, gb);
      for (int v = 0; v < V; ++v) gb[v] = fmaf(a[v], gb[v], b[v]), ga[v] *= a[v];
      publish<V>(p.ends, index, p.width, c, ga, gb);
    }
    if (w < groups || (w == W - 1 && place > run)) {
      const int back = w < groups ? behind + 1 + W * (groups - 1 - w) : run + 1;
      wait_for<V>(p.ends, index - static_cast<int64_t>(ahead) * back, p.width, c, a, b);
      write<V>(s.groups[w], lane, a, b);
    }
    __syncthreads();
    if (place > run) apply<V>(s.groups[W - 1], lane, h);
    for (int k = 0; k < groups; ++k) apply<V>(s.groups[k], lane, h);
    for (int k = 0; k < behind; ++k) apply<V>(s.pieces[k], lane, h);
  }
  for (int k = 0; k < w; ++k) apply<V>(s.own[k], lane, h);
  for (int v = 0; v < V; ++v) end[v] = h[v];
  if (w == W - 1) {
    apply<V>(s.own[W - 1], lane, end);
    if (LINKED && run == W * W - 1) {
      float none[V];
      for (int v = 0; v < V; ++v) none[v] = 0.0f;
      publish<V>(p.ends, index, p.width, c, none, end);
    }
  }
}

// The piece and channels of this workgroup; direction -1 takes pieces from the last to the first.
template <int V, int W, bool LINKED>
__device__ __forceinline__ int64_t next_piece(const ScanArgs& p, Shared<V, W>& s, int direction, int& block) {
  uint32_t id = blockIdx.x;
  if (LINKED) {
    // the ticket starts at 2^32 - 1, as the clearing leaves it
    if (threadIdx.x == 0) s.ticket = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u;
    __syncthreads();
    id = __builtin_amdgcn_readfirstlane(s.ticket);
  }
  block = static_cast<int>(id % static_cast<uint32_t>(p.blocks));
  const int64_t piece = id / static_cast<uint32_t>(p.blocks);
  return direction > 0 ? piece : p.pieces - 1 - piece;
}

// A piece of no request hands on nothing, but nobody may wait for it.
template <int V, bool LINKED>
__device__ __forceinline__ void publish_nothing(const ScanArgs& p, int64_t index, int w, int c) {
  if (!LINKED || w != 0) return;
  float a[V], b[V];
  for (int v = 0; v < V; ++v) a[v] = 1.0f, b[v] = 0.0f;
  publish<V>(p.maps, index, p.width, c, a, b);
  publish<V>(p.ends, index, p.width, c, a, b);
}

template <int V, bool LINKED>
__device__ __forceinline__ void load_speeds(const ScanArgs& p, int c, float (&speed)[V]) {
  for (int v = 0; v < V; ++v) speed[v] = LINKED ? p.speeds[c + v] : speed_of(p.decay[c + v], p.rate);
}

// One workgroup takes a piece of a request, 64 V channels of it: 96 loads of 4 bytes a lane are under way at once, 12
// waves a compute unit.  One prompt of 32768 x 4096 bfloat16 takes 234 us, 4.6 TB/s (a copy of its bytes 208): 35 vector
// instructions an element, 5 of them of half rate, are 137 us of all vector units, which the loads hide in part.
// Two channels a lane where 16-bit rows allow it, single ones otherwise (3001 x 1001 binary32: 18.6 us).
template <typename T, int V, bool LINKED, int R, int W>
__global__ void __launch_bounds__(64 * W) k_scan(ScanArgs p) {
  constexpr int kPiece = R * W;
  __shared__ Shared<V, W> s;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int block;
  const int64_t index = next_piece<V, W, LINKED>(p, s, 1, block);
  const Piece q = find<kPiece>(p, index);
  const int c = (block * 64 + lane) * V;
  if (q.request < 0) return publish_nothing<V, LINKED>(p, index, w, c);
  const bool mine = c < p.width;
  const uint32_t cc = mine ? c : 0;
  const int slot = slot_of(p, q.request);
  const int64_t t0 = q.first + static_cast<int64_t>(q.tile) * kPiece + w * R;
  const int n = max(0, min(R, q.count - q.tile * kPiece - w * R));
  float a[R][V], u[R][V], A[V], B[V], h[V], end[V];
  for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f;
  // every loop over tokens has to be unrolled, or what it fills is not in registers
  const auto read = [&](auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
    float speed[V];
    load_speeds<V, LINKED>(p, cc, speed);
    Vec<T, V> xr[R], gr[R], ir[R];
    const Rows<T, V> x(p.x, p.x_stride, t0, cc), ga(p.ga, p.ga_stride, t0, cc), gx(p.gx, p.gx_stride, t0, cc);
#pragma unroll
    for (int t = 0; t < R; ++t) {                 // rows behind the last one are read as it
      const int row = WHOLE ? t : min(t, n - 1);
      xr[t] = x.load(row);
      gr[t] = ga.load(row);
      ir[t] = gx.load(row);
    }
#pragma unroll
    for (int t = 0; t < R; ++t)
      for (int v = 0; v < V; ++v) {
        const float less = one_less_exp2(speed[v] * logistic(gr[t][v]));
        const float keep = 1.0f - less;
        const float in = __builtin_amdgcn_sqrtf(less * (1.0f + keep)) * logistic(ir[t][v]) * xr[t][v];
        a[t][v] = WHOLE || t < n ? keep : 1.0f;
        u[t][v] = WHOLE || t < n ? in : 0.0f;
        A[v] *= a[t][v], B[v] = fmaf(a[t][v], B[v], u[t][v]);
      }
  };
  if (n == R) {
    read(std::true_type{});
  } else {
#pragma unroll
    for (int t = 0; t < R; ++t)
      for (int v = 0; v < V; ++v) a[t][v] = 1.0f, u[t][v] = 0.0f;
    if (n > 0) read(std::false_type{});
  }
  state_of<V>(p, slot, q.tile == 0 && slot >= 0 && p.resume != nullptr && p.resume[q.request] != 0, cc, h);
  if (slot == -2)
    for (int v = 0; v < V; ++v) h[v] = __builtin_nanf("");
  hand_on<V, W, LINKED>(p, s, w, lane, index, 1, q.tile, c, A, B, h, end);
  if (!mine) return;
  // as find() does for pieces: the states before every kBackTokens tokens
  const Rows<T, V> y(p.y, p.y_stride, t0, cc);
  const int64_t saved0 = q.first / kBackTokens + q.request + (q.tile * W + w) * (R / kBackTokens);
  float* saved = p.saved == nullptr ? nullptr : p.saved + saved0 * p.width + cc;
#pragma unroll
  for (int t = 0; t < R; ++t) {
    if (t % kBackTokens == 0 && t < n && saved != nullptr)
      for (int v = 0; v < V; ++v) saved[t / kBackTokens * static_cast<int64_t>(p.width) + v] = h[v];
    for (int v = 0; v < V; ++v) h[v] = fmaf(a[t][v], h[v], u[t][v]);
    if (t < n) y.store(t, h);
  }
  if (w == W - 1 && slot >= 0 && static_cast<int64_t>(q.tile + 1) * kPiece >= q.count)
    for (int v = 0; v < V; ++v) p.state[static_cast<int64_t>(slot) * p.width + c + v] = h[v];
}

// Two workgroups a compute unit (128 registers a lane; with 140 there is one, 352 us for the training step below).
// 12288 tokens x 4096 bfloat16 take 190 us, 3.7 TB/s (the floor is 136): 77 vector instructions an element, vector units
// 68 % busy, waves wait 53 % of their time, for loads that the other workgroup's work does not cover.
template <typename T, int V, bool LINKED>
__global__ void __launch_bounds__(64 * kBackWaves, 4) k_scan_backward(ScanArgs p) {
  constexpr int R = kBackTokens, W = kBackWaves;
  __shared__ Shared<V, W> s;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int block;
  const int64_t index = next_piece<V, W, LINKED>(p, s, -1, block);
  const Piece q = find<kBackPiece>(p, index);
  const int c = (block * 64 + lane) * V;
  const bool mine = c < p.width;
  if (q.request < 0) {
    if (w == 0 && mine)
      for (int v = 0; v < V; ++v) p.partial[index * p.width + c + v] = 0.0f;
    return publish_nothing<V, LINKED>(p, index, w, c);
  }
  const uint32_t cc = mine ? c : 0;
  const int slot = slot_of(p, q.request);
  // wave 0 holds the last tokens: it is the first that the gradients reach
  const int back = W - 1 - w;
  const int64_t t0 = q.first + static_cast<int64_t>(q.tile) * kBackPiece + back * R;
  const int n = max(0, min(R, q.count - q.tile * kBackPiece - back * R));
  const int last = q.count > 0 ? (q.count - 1) / kBackPiece : 0;
  float less[R][V], A[V], B[V], g[V], end[V], speed[V], sum[V];
  Vec<T, V> ar[R], gr[R], xr[R], ir[R];
  for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f, sum[v] = 0.0f;
  const auto read = [&](auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
    load_speeds<V, LINKED>(p, cc, speed);
    if (slot == -2)                                 // makes every gradient NaN
      for (int v = 0; v < V; ++v) speed[v] = __builtin_nanf("");
    const Rows<T, V> x(p.x, p.x_stride, t0, cc), ga(p.ga, p.ga_stride, t0, cc), gx(p.gx, p.gx_stride, t0, cc);
    const Rows<T, V> dy(p.dy, p.dy_stride, t0, cc);
    // in the order of their use; rows behind the last one are read as it
#pragma unroll
    for (int t = R - 1; t >= 0; --t) {
      const int row = WHOLE ? t : min(t, n - 1);
      ar[t] = ga.load(row);
      gr[t] = dy.load(row);
    }
#pragma unroll
    for (int t = 0; t < R; ++t) {
      const int row = WHOLE ? t : min(t, n - 1);
      xr[t] = x.load(row);
      ir[t] = gx.load(row);
    }
#pragma unroll
    for (int t = R - 1; t >= 0; --t)
      for (int v = 0; v < V; ++v) {
        less[t][v] = one_less_exp2(speed[v] * logistic(ar[t][v]));
        if (WHOLE || t < n) {
          const float keep = 1.0f - less[t][v];
          A[v] *= keep, B[v] = keep * (B[v] + gr[t][v]);
        }
      }
  };
  if (n == R) read(std::true_type{});
  else if (n > 0) read(std::false_type{});
  state_of<V>(p, slot, slot >= 0 && q.tile == last, cc, g);
  hand_on<V, W, LINKED>(p, s, w, lane, index, -1, last - q.tile, c, A, B, g, end);
  // The gates are worked out again from what was read rather than kept: registers are what limits how many
  // workgroups a compute unit has under way.
  const auto gradients = [&](auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
    const Rows<T, V> dx(p.y, p.y_stride, t0, cc), dga(p.dga, p.dga_stride, t0, cc), dgx(p.dgx, p.dgx_stride, t0, cc);
    float before[R][V], h[V], slow[V];
    for (int v = 0; v < V; ++v) {
      h[v] = p.saved[(q.first / R + q.request + q.tile * W + back) * p.width + cc + v];
      slow[v] = speed[v] * kLog2;
    }
#pragma unroll
    for (int t = 0; t < R; ++t) {
      for (int v = 0; v < V; ++v) {
        const float a = 1.0f - less[t][v];
        before[t][v] = h[v];
        h[v] = fmaf(a, h[v], __builtin_amdgcn_sqrtf(less[t][v] * (1.0f + a)) * logistic(ir[t][v]) * xr[t][v]);
      }
      again(ir[t]), again(xr[t]);
    }
#pragma unroll
    for (int t = R - 1; t >= 0; --t) {
      if (!WHOLE && t >= n) continue;
      float ox[V], oa[V], oi[V];
      for (int v = 0; v < V; ++v) {
        const float a = 1.0f - less[t][v], b2 = less[t][v] * (1.0f + a);
        // a state that is kept whole has no slope; the reciprocal root of a number below the normal ones is infinite
        const float inv = b2 >= 1.17549435e-38f ? __builtin_amdgcn_rsqf(b2) : 0.0f;
        const float ra = logistic(ar[t][v]), ri = logistic(ir[t][v]);
        const float gain = ri * xr[t][v];
        const float now = g[v] + gr[t][v], in = now * (b2 * inv);
        g[v] = a * now;
        const float P = g[v] * (slow[v] * ra) * fmaf(-a, gain * inv, before[t][v]);
        ox[v] = in * ri;
        oi[v] = in * gain * (1.0f - ri);
        oa[v] = P * (1.0f - ra);
        sum[v] += P;
      }
      if (mine) {
        dx.store(t, ox);
        dga.store(t, oa);
        dgx.store(t, oi);
      }
    }
  };
  if (n == R) gradients(std::true_type{});
  else if (n > 0) gradients(std::false_type{});
  if (slot == -2)
    for (int v = 0; v < V; ++v) sum[v] = 0.0f;
  if (w == W - 1 && slot >= 0 && q.tile == 0 && mine)
    for (int v = 0; v < V; ++v)
      p.state[static_cast<int64_t>(slot) * p.width + c + v] = p.resume != nullptr && p.resume[q.request] != 0 ? end[v] : 0.0f;
  // a sum over the piece, the waves in order
  __syncthreads();
  write<V>(s.own[w], lane, sum, sum);
  __syncthreads();
  if (w != 0 || !mine) return;
  for (int v = 0; v < V; ++v) {
    float all = 0.0f;
    for (int k = 0; k < W; ++k) all += s.own[k][0][lane * V + v];
    p.partial[index * p.width + c + v] = all;
  }
}

// ddecay from the pieces' parts, added in order in binary64: a wave takes 64 channels and
// every 16th piece: 7 us for 198 pieces of 4096 channels.
__global__ void __launch_bounds__(1024) k_scan_decay(ScanArgs p) {
  __shared__ double sums[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  double sum = 0.0;
  if (c < p.width)
    for (int64_t j = w; j < p.pieces; j += 128) {
      float x[8];                     // under way together
      for (int i = 0; i < 8; ++i) x[i] = j + 16 * i < p.pieces ? p.partial[(j + 16 * i) * p.width + c] : 0.0f;
      for (int i = 0; i < 8; ++i) sum += x[i];
    }
  sums[w][lane] = sum;
  __syncthreads();
  if (w != 0 || c >= p.width) return;
  for (int s = 1; s < 16; ++s) sum += sums[s][lane];
  // s(decay) / softplus(decay) goes to 1 where both vanish
  const double e = exp(-fabs(static_cast<double>(p.decay[c]))), d = p.decay[c];
  const double soft = (d > 0.0 ? d : 0.0) + log1p(e), open = d > 0.0 ? 1.0 / (1.0 + e) : e / (1.0 + e);
  p.ddecay[c] = static_cast<float>(soft > 0.0 ? sum * (open / soft) : sum);
}

// Bound by memory: 512 requests of 6144 bfloat16 channels take 10.4 us, 4.9 TB/s (a copy of their
// bytes 9.8).  Where there are many, a
// lane takes its channels of `rows` requests, one behind the other, and works out the decay's speed once.
template <typename T, int V>
__global__ void __launch_bounds__(256) k_scan_step(ScanArgs p, int rows) {
  const int groups = (p.width + 256 * V - 1) / (256 * V);
  const int b0 = static_cast<int>(blockIdx.x / groups) * rows;
  const int c = (static_cast<int>(blockIdx.x % groups) * 256 + static_cast<int>(threadIdx.x)) * V;
  if (c >= p.width) return;
  float speed[V];
  for (int v = 0; v < V; ++v) speed[v] = speed_of(p.decay[c + v], p.rate);
  for (int b = b0; b < min(b0 + rows, p.batch); ++b) {
    const int slot = p.slot_ids[b];
    float h[V];
    if (slot < 0 || slot >= p.num_slots) {
      for (int v = 0; v < V; ++v) h[v] = __builtin_nanf("");
      store<T, V>(static_cast<T*>(p.y) + b * p.y_stride + c, h);
      continue;
    }
    const Vec<T, V> xr = load<T, V>(static_cast<const T*>(p.x) + b * p.x_stride + c),
                    gr = load<T, V>(static_cast<const T*>(p.ga) + b * p.ga_stride + c),
                    ir = load<T, V>(static_cast<const T*>(p.gx) + b * p.gx_stride + c);
    float* at = p.state + static_cast<int64_t>(slot) * p.width + c;
    for (int v = 0; v < V; ++v) {
      const float less = one_less_exp2(speed[v] * logistic(gr[v]));
      const float a = 1.0f - less;
      h[v] = fmaf(a, at[v], __builtin_amdgcn_sqrtf(less * (1.0f + a)) * logistic(ir[v]) * xr[v]);
    }
    for (int v = 0; v < V; ++v) at[v] = h[v];
    store<T, V>(static_cast<T*>(p.y) + b * p.y_stride + c, h);
  }
}

// Two channels a lane where values have 16 bits and every pair lies on a boundary of its size.  Binary32 pairs take twice the
// registers for what is read: 18391 tokens x 1408, us of forward and backward, 102 and 215 in pairs, 103 and 164 one by one.
bool in_pairs(const ScanArgs& a, int esize) {
  const auto pair = [&](const void* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % (2 * esize) == 0 && stride % 2 == 0;
  };
  return esize == 2 && a.width % 2 == 0 && pair(a.x, a.x_stride) && pair(a.ga, a.ga_stride) && pair(a.gx, a.gx_stride) &&
         pair(a.y, a.y_stride) && pair(a.dy, a.dy_stride) && pair(a.dga, a.dga_stride) && pair(a.dgx, a.dgx_stride);
}

// Every piece's workgroups, behind the clearing of the words that they hand on.
template <typename T, bool BACK>
hipError_t over_pieces(ScanArgs a, hipStream_t s) {
  const bool two = in_pairs(a, sizeof(T)), linked = a.ticket != nullptr;
  a.blocks = two ? (a.width + 127) / 128 : (a.width + 63) / 64;
  if (linked) {
    const int64_t all = (a.words + 255) / 256;
    k_scan_clear<<<dim3(static_cast<uint32_t>(all < 1024 ? all : 1024)), 256, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid(static_cast<uint32_t>(static_cast<int64_t>(a.pieces) * a.blocks));
  const auto go = [&](auto v, auto l) {
    constexpr int V = decltype(v)::value;
    constexpr bool LINKED = decltype(l)::value;
    if constexpr (BACK) {
      k_scan_backward<T, V, LINKED><<<grid, 64 * kBackWaves, 0, s>>>(a);
    } else if (a.piece == kFewPiece) {
      k_scan<T, V, LINKED, kFewTokens, kFewWaves><<<grid, 64 * kFewWaves, 0, s>>>(a);
    } else {
      k_scan<T, V, LINKED, kScanTokens, kScanWaves><<<grid, 64 * kScanWaves, 0, s>>>(a);
    }
  };
  const std::integral_constant<int, 1> one{};
  const std::integral_constant<int, 2> pair{};
  if (!two) linked ? go(one, std::true_type{}) : go(one, std::false_type{});
  else if constexpr (sizeof(T) == 2) linked ? go(pair, std::true_type{}) : go(pair, std::false_type{});
  return hipGetLastError();
}

template <typename T>
hipError_t forward(const ScanArgs& a, hipStream_t s) { return over_pieces<T, false>(a, s); }

template <typename T>
hipError_t backward(const ScanArgs& a, hipStream_t s) {
  if (a.pieces > 0) {
    const hipError_t e = over_pieces<T, true>(a, s);
    if (e != hipSuccess) return e;
  }
  k_scan_decay<<<dim3(static_cast<uint32_t>((a.width + 63) / 64)), 1024, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t step(const ScanArgs& a, hipStream_t s) {
  const bool two = in_pairs(a, sizeof(T));
  const int channels = two ? 512 : 256;
  const int64_t groups = (a.width + channels - 1) / channels;
  // us of 1, 2, 4 and 8 requests a workgroup, by workgroups of the former (bfloat16, 6144 channels): 768 3.6, 3.6, 4.2, 5.9;  1536 4.4,
  // 4.3, 4.9, 6.2;  4080 7.8, 7.0, 6.7, 7.9;  6144 11.9, 10.3, 9.7, 11.4;  12288 21.1, 18.6, 18.0, 18.0.  Of 1001 channels one by one:
  // 2048 4.4, 4.2, 4.4, 5.5;  8192 10.3, 8.3, 7.4, 8.0
  const int rows = groups * a.batch >= 4096 ? 4 : 1;
  const dim3 grid(static_cast<uint32_t>((a.batch + rows - 1) / rows * groups));
  if (!two) k_scan_step<T, 1><<<grid, 256, 0, s>>>(a, rows);
  else if constexpr (sizeof(T) == 2) k_scan_step<T, 2><<<grid, 256, 0, s>>>(a, rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_forward(const ScanArgs& a, int dtype, hipStream_t s) {
  return dtype == STEPQ_BF16 ? forward<__bf16>(a, s) : dtype == STEPQ_F16 ? forward<_Float16>(a, s) : forward<float>(a, s);
}
hipError_t launch_scan_backward(const ScanArgs& a, int dtype, hipStream_t s) {
  return dtype == STEPQ_BF16 ? backward<__bf16>(a, s) : dtype == STEPQ_F16 ? backward<_Float16>(a, s) : backward<float>(a, s);
}
hipError_t launch_scan_step(const ScanArgs& a, int dtype, hipStream_t s) {
  return dtype == STEPQ_BF16 ? step<__bf16>(a, s) : dtype == STEPQ_F16 ? step<_Float16>(a, s) : step<float>(a, s);
}

}  // namespace stepq
