// gfx950 kernels of the norms around a block, forward and backward.
//
// A row is shared by `L` lanes, each of which holds `P` pieces of 16 bytes of every
// tensor of it in registers from the load to the store: every tensor is read or written
// once, and a row's two sums (of o^2, then of t^2, which depends on the first) are the only
// exchange.  The same lane reads and writes an element, so outputs may lie where inputs did.
// A backward pass of more than 4096 values has several pieces a lane, and no registers for all of them: what goes to
// scratch memory and back makes 4096 tokens of 8192 bfloat16 values 152 us where a copy of their bytes takes 104, 2048 of
// 16384 665.
//
// Backward, with r1 and r2 the reciprocal roots, p = n act(z) and v = pre_weight dy:
//   gt = dt + r2 v - t r2^3 mean(t v)       the gradient of t, and of the residual
//   dscale = sum gt p,  q = scale gt,  dz = q n act'(z),  m = q act(z)
//   dpost = sum m o r1,  do = r1 w m - o r1^3 mean(o w m),  dpre = sum dy t r2
// The weights' gradients are summed over a workgroup's rows in registers, over workgroups
// in a second launch, in order.
#include <type_traits>

#include "norm_internal.hpp"

namespace stepq {
namespace {

// Workgroups of a forward pass: each takes several rows, so that weights are read once for them.  us of 8192
// tokens of 4096, of 8192 x 48 rows of 128: 1024 workgroups 73, 58; 2048 79, 65; one a row 217, 133.
constexpr int kGrid = 1024;
constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
constexpr int kVec = 16 / sizeof(T);

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// As it lies in memory until it is used: 16-bit pairs stay in one register.
template <typename T>
struct Piece {
  u32x4 raw;
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(T) == 4) {
      return __builtin_bit_cast(float, static_cast<uint32_t>(raw[i]));
    } else {
      const uint32_t w = raw[i / 2];
      if constexpr (std::is_same<T, __bf16>::value) return __builtin_bit_cast(float, i % 2 ? w & 0xffff0000u : w << 16);
      else return static_cast<float>(__builtin_bit_cast(T, static_cast<uint16_t>(i % 2 ? w >> 16 : w)));
    }
  }
};
template <typename T>
__device__ __forceinline__ u32x4 rounded(const float (&x)[kVec<T>]) {
  typedef T Some __attribute__((ext_vector_type(kVec<T>)));
  Some r;
  for (int i = 0; i < kVec<T>; ++i) r[i] = static_cast<T>(x[i]);
  return __builtin_bit_cast(u32x4, r);
}

// 16 bytes on the boundary of an element: the memory system takes them whole, a cache line more at worst.
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Anywhere {
  u32x4 raw;
};

// The values at .. of a row, zeros behind its end.  IN16: rows lie on 16-byte boundaries and hold whole
// pieces.  us of 8192 bfloat16 tokens of 1001, forward and backward, with single elements 52, 97, with 16 bytes
// anywhere 22, 64 (now 22, 57).
template <typename T, bool IN16>
__device__ __forceinline__ Piece<T> load(const T* row, int at, int width) {
  if constexpr (IN16) {
    Piece<T> r = {u32x4{0, 0, 0, 0}};
    if (at < width) r.raw = *reinterpret_cast<const u32x4*>(row + at);
    return r;
  } else {
    if (at + kVec<T> <= width) return {reinterpret_cast<const Anywhere<T>*>(row + at)->raw};
    typedef T Some __attribute__((ext_vector_type(kVec<T>)));
    Some r;
    for (int i = 0; i < kVec<T>; ++i) r[i] = at + i < width ? row[at + i] : static_cast<T>(0.0f);
    return {__builtin_bit_cast(u32x4, r)};
  }
}
template <typename T, bool IN16>
__device__ __forceinline__ void store(T* row, int at, int width, const float (&x)[kVec<T>]) {
  if constexpr (IN16) {
    if (at < width) *reinterpret_cast<u32x4*>(row + at) = rounded<T>(x);
  } else if (at + kVec<T> <= width) {
    reinterpret_cast<Anywhere<T>*>(row + at)->raw = rounded<T>(x);
  } else {
    for (int i = 0; i < kVec<T>; ++i)
      if (at + i < width) row[at + i] = static_cast<T>(x[i]);
  }
}

template <int CTRL>
__device__ __forceinline__ float moved(float x) {
  const int i = __builtin_bit_cast(int, x);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, CTRL, 0xf, 0xf, false));
}

// Sums over the L lanes of a row, the same bits in each of them: at every step both of two lanes add what the other
// one has, and lanes whose sums are of the same values have the same bits of them.
template <int L, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float (*lds)[N]) {
  for (int n = 0; n < N; ++n) {
    x[n] += moved<0xB1>(x[n]);          // quad_perm: neighbours, then pairs
    x[n] += moved<0x4E>(x[n]);
    if (L >= 16) {
      x[n] += moved<0x141>(x[n]);       // row_half_mirror: the other four of eight, row_mirror: the other eight of sixteen
      x[n] += moved<0x140>(x[n]);
    }
    if (L >= 64) {
      x[n] += __shfl_xor(x[n], 16);
      x[n] += __shfl_xor(x[n], 32);
    }
  }
  if (L > 64) {
    const int w = threadIdx.x >> 6, first = threadIdx.x / L * (L / 64);
    if ((threadIdx.x & 63) == 0)
      for (int n = 0; n < N; ++n) lds[w][n] = x[n];
    __syncthreads();
    for (int n = 0; n < N; ++n) {
      float all = lds[first][n];
      for (int s = 1; s < L / 64; ++s) all += lds[first + s][n];
      x[n] = all;
    }
  }
}

__device__ __forceinline__ float logistic(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// act(z) and, where it is asked for, its slope.  A gate of -inf shuts.
__device__ __forceinline__ float activated(float z, bool silu) {
  const float s = logistic(z);
  return !silu ? s : s == 0.0f ? 0.0f : z * s;
}
__device__ __forceinline__ float activated(float z, bool silu, float& slope) {
  const float s = logistic(z), rest = 1.0f - s;
  if (!silu) return slope = s * rest, s;
  const float bend = rest == 0.0f || s == 0.0f ? 0.0f : z * rest;
  slope = s * (1.0f + bend);
  return s == 0.0f ? 0.0f : z * s;
}

template <typename T>
__device__ __forceinline__ const T* row_of(const NormRows& r, int row, int heads, int width) {
  const T* p = static_cast<const T*>(r.p);
  if (heads == 1) return p + row * r.stride;
  const uint32_t token = static_cast<uint32_t>(row) / static_cast<uint32_t>(heads);
  return p + token * r.stride + static_cast<int64_t>(row - token * heads) * width;
}
template <typename T>
__device__ __forceinline__ T* out_row_of(const NormRows& r, int row, int heads, int width) {
  return const_cast<T*>(row_of<T>(r, row, heads, width));
}

// A lane's part of a weight, 1 where there is none and behind the row's end.
template <typename T, int P>
__device__ __forceinline__ void load_weight(float (&w)[P][kVec<T>], const float* from, int lane, int L, int width) {
  for (int j = 0; j < P; ++j) {
    const int at = (j * L + lane) * kVec<T>;
    if (from != nullptr && at + kVec<T> <= width) {
      for (int i = 0; i < kVec<T>; i += 4) {
        const u32x4 r = reinterpret_cast<const Anywhere<float>*>(from + at + i)->raw;
        for (int k = 0; k < 4; ++k) w[j][i + k] = __builtin_bit_cast(float, static_cast<uint32_t>(r[k]));
      }
    } else {
      for (int i = 0; i < kVec<T>; ++i) w[j][i] = from != nullptr && at + i < width ? from[at + i] : 1.0f;
    }
  }
}

constexpr int threads_of(int L) { return L < kNormThreads ? kNormThreads : L; }
constexpr int at_once(int L) { return threads_of(L) / L; }

// What of a row a group of L lanes reads: nothing behind the last row, since another group may be writing an output
// where its inputs were.  A workgroup of one group has a row whenever it looks for one.
template <int L>
__device__ __forceinline__ int width_of(int64_t row, const NormArgs& p) {
  if constexpr (at_once(L) == 1) return p.width;
  const int width = row < p.rows ? p.width : 0;
  return L >= 64 ? __builtin_amdgcn_readfirstlane(width) : width;
}

// to + a b where the group has a row.  Behind the last one a product may be NaN, by a weight that is infinite.
template <int L>
__device__ __forceinline__ float added(bool real, float a, float b, float to) {
  if constexpr (at_once(L) == 1) return fmaf(real ? a : 0.0f, b, to);
  else return real ? fmaf(a, b, to) : to;
}

// The pieces of a row of `width` values that a lane holds.
template <typename T, bool IN16, int L, int P>
__device__ __forceinline__ void load_row(const NormRows& r, int row, const NormArgs& p, int lane, int width, Piece<T> (&x)[P]) {
  if (r.p == nullptr) return;
  const T* at = row_of<T>(r, row, p.heads, p.width);
  for (int j = 0; j < P; ++j) x[j] = load<T, IN16>(at, (j * L + lane) * kVec<T>, width);
}

// Bound by memory: 8192 tokens of 4096 bfloat16 values, all parts, take 65 us, 5.2 TB/s, 8192 x 48 gated rows of 128 57.6,
// both at the rate of a copy.  16-bit pairs stay in one register until they are used, which leaves room for four
// workgroups a compute unit and the next row ahead (114 and 80 us before either).
template <typename T, bool IN16, int L, int P>
__global__ void __launch_bounds__(threads_of(L)) k_norm(NormArgs p) {
  constexpr int V = kVec<T>, kAtOnce = at_once(L);
  __shared__ float lds[2][threads_of(L) / 64][1];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const float inv = 1.0f / static_cast<float>(p.width);
  float w1[P][V], sc[P][V], w2[P][V];
  load_weight<T, P>(w1, p.post_weight, lane, L, p.width);
  load_weight<T, P>(sc, p.scale, lane, L, p.width);
  load_weight<T, P>(w2, p.pre_weight, lane, L, p.width);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kAtOnce, first0 = static_cast<int64_t>(blockIdx.x) * kAtOnce;
  Piece<T> o[P], z[P], x[P];
  const auto read = [&](int64_t first) {
    const int row = static_cast<int>(first + group < p.rows ? first + group : p.rows - 1);
    const int width = width_of<L>(first + group, p);
    load_row<T, IN16, L, P>(p.block, row, p, lane, width, o);
    load_row<T, IN16, L, P>(p.gate, row, p, lane, width, z);
    load_row<T, IN16, L, P>(p.residual, row, p, lane, width, x);
  };
  if (first0 < p.rows) read(first0);
  for (int64_t first = first0; first < p.rows; first += step) {
    const bool real = first + group < p.rows;
    const int row = static_cast<int>(real ? first + group : p.rows - 1);
    float r1 = 1.0f;
    if (p.post) {
      float s[1] = {0.0f};
      for (int j = 0; j < P; ++j)
        for (int i = 0; i < V; ++i) s[0] = fmaf(o[j][i], o[j][i], s[0]);
      row_sums<L>(s, lds[0]);
      r1 = __builtin_amdgcn_rsqf(fmaf(s[0], inv, p.eps));
    }
    float t[P][V], s[1] = {0.0f};
    for (int j = 0; j < P; ++j)
      for (int i = 0; i < V; ++i) {
        float g = o[j][i] * r1 * w1[j][i];
        if (p.gate.p != nullptr) g *= activated(z[j][i], p.silu);
        t[j][i] = p.residual.p != nullptr ? fmaf(sc[j][i], g, x[j][i]) : sc[j][i] * g;
        s[0] = fmaf(t[j][i], t[j][i], s[0]);
      }
    if (first + step < p.rows) read(first + step);      // in flight while this row ends
    if (p.out.p != nullptr && real)
      for (int j = 0; j < P; ++j)
        store<T, IN16>(out_row_of<T>(p.out, row, p.heads, p.width), (j * L + lane) * V, p.width, t[j]);
    if (p.pre) {
      row_sums<L>(s, lds[1]);
      const float r2 = __builtin_amdgcn_rsqf(fmaf(s[0], inv, p.eps));
      for (int j = 0; j < P; ++j) {
        float y[V];
        for (int i = 0; i < V; ++i) y[i] = t[j][i] * r2 * w2[j][i];
        if (real) store<T, IN16>(out_row_of<T>(p.normed, row, p.heads, p.width), (j * L + lane) * V, p.width, y);
      }
    }
    // the next row's sums overwrite this one's, which were read before the other sum's barrier
    if (L > 64 && !(p.post && p.pre)) __syncthreads();
  }
}

// 8192 tokens of 4096 bfloat16 values, all parts, take 120 us, 4.5 TB/s (a copy of their bytes 104): one workgroup of 512 lanes a
// compute unit, whose 160 registers hold the weights, their gradients and the next row, vector units 61 % busy.
template <typename T, bool IN16, int L, int P>
__global__ void __launch_bounds__(threads_of(L)) k_norm_backward(NormArgs p) {
  constexpr int V = kVec<T>, kAtOnce = at_once(L), kThreads = threads_of(L);
  __shared__ float lds1[kThreads / 64][3];
  __shared__ float lds2[kThreads / 64][1];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const float inv = 1.0f / static_cast<float>(p.width);
  float w1[P][V], sc[P][V], w2[P][V], d1[P][V], ds[P][V], d2[P][V];
  const auto weights = [&]() {
    load_weight<T, P>(w1, p.post_weight, lane, L, p.width);
    load_weight<T, P>(sc, p.scale, lane, L, p.width);
    load_weight<T, P>(w2, p.pre_weight, lane, L, p.width);
  };
  // lanes with several pieces have no room to keep the weights too, every row reads them again: 4096 tokens
  // of 8192 bfloat16 values 155 us against 294
  constexpr bool kAgain = P > 1;
  if (!kAgain) weights();
  for (int j = 0; j < P; ++j)
    for (int i = 0; i < V; ++i) d1[j][i] = ds[j][i] = d2[j][i] = 0.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kAtOnce, first0 = static_cast<int64_t>(blockIdx.x) * kAtOnce;
  Piece<T> o[P], z[P], t[P], gt[P], gy[P];
  const auto read = [&](int64_t first) {
    const int row = static_cast<int>(first + group < p.rows ? first + group : p.rows - 1);
    const int width = width_of<L>(first + group, p);
    load_row<T, IN16, L, P>(p.block, row, p, lane, width, o);
    load_row<T, IN16, L, P>(p.gate, row, p, lane, width, z);
    load_row<T, IN16, L, P>(p.d_out, row, p, lane, width, gt);
    load_row<T, IN16, L, P>(p.out, row, p, lane, width, t);
    load_row<T, IN16, L, P>(p.d_normed, row, p, lane, width, gy);
  };
  if (first0 < p.rows) read(first0);
  for (int64_t first = first0; first < p.rows; first += step) {
    const bool real = first + group < p.rows;
    const int row = static_cast<int>(real ? first + group : p.rows - 1);
    if (kAgain) weights();
    float s[3] = {0.0f, 0.0f, 0.0f};
    for (int j = 0; j < P; ++j)
      for (int i = 0; i < V; ++i) {
        const float a = o[j][i];
        s[0] = fmaf(a, a, s[0]);
        if (p.pre) {
          const float b = t[j][i];
          s[1] = fmaf(b, b, s[1]);
          s[2] = fmaf(b, w2[j][i] * gy[j][i], s[2]);
        }
      }
    row_sums<L>(s, lds1);
    const float r1 = p.post ? __builtin_amdgcn_rsqf(fmaf(s[0], inv, p.eps)) : 1.0f;
    const float r2 = __builtin_amdgcn_rsqf(fmaf(s[1], inv, p.eps)), back = s[2] * inv * r2 * r2;
    float m[P][V], sum[1] = {0.0f};
    Piece<T> keep[P];
    for (int j = 0; j < P; ++j) {
      float all[V], dz[V];
      for (int i = 0; i < V; ++i) {
        float g = p.d_out.p != nullptr ? gt[j][i] : 0.0f;
        if (p.pre) {
          const float b = t[j][i], dy = gy[j][i];
          g += r2 * (w2[j][i] * dy - b * back);
          d2[j][i] = added<L>(real, dy, b * r2, d2[j][i]);
        }
        all[i] = g;
        const float u = o[j][i] * r1, n = u * w1[j][i];
        float slope = 0.0f, act = 1.0f;
        if (p.gate.p != nullptr) act = activated(z[j][i], p.silu, slope);
        ds[j][i] = added<L>(real, g, n * act, ds[j][i]);
        const float q = g * sc[j][i];
        dz[i] = q * n * slope;
        const float k = q * act;
        d1[j][i] = added<L>(real, k, u, d1[j][i]);
        m[j][i] = k * w1[j][i];
        sum[0] = fmaf(o[j][i], m[j][i], sum[0]);
      }
      const int at = (j * L + lane) * V;
      if (p.d_residual.p != nullptr && real) store<T, IN16>(out_row_of<T>(p.d_residual, row, p.heads, p.width), at, p.width, all);
      if (p.gate.p != nullptr && real) store<T, IN16>(out_row_of<T>(p.d_gate, row, p.heads, p.width), at, p.width, dz);
      keep[j] = o[j];
    }
    if (first + step < p.rows) read(first + step);      // in flight while this row ends
    row_sums<L>(sum, lds2);
    const float mean = p.post ? sum[0] * inv * r1 * r1 : 0.0f;
    for (int j = 0; j < P; ++j) {
      float d[V];
      for (int i = 0; i < V; ++i) d[i] = r1 * (m[j][i] - keep[j][i] * mean);
      if (real) store<T, IN16>(out_row_of<T>(p.d_block, row, p.heads, p.width), (j * L + lane) * V, p.width, d);
    }
  }
  if (p.partial == nullptr) return;
  // the workgroup's rows that were under way together are added in order
  constexpr int kSlots = kAtOnce > 1 ? kThreads * V * P : 1;
  __shared__ float part[kSlots];
  for (int k = 0; k < 3; ++k) {
    float(&d)[P][V] = k == 0 ? d1 : k == 1 ? ds : d2;
    float* to = p.partial + (static_cast<int64_t>(k) * p.groups + blockIdx.x) * p.width;
    if (kAtOnce > 1) {
      __syncthreads();
      for (int j = 0; j < P; ++j)
        for (int i = 0; i < V; ++i) part[group * (L * V * P) + (j * L + lane) * V + i] = d[j][i];
      __syncthreads();
      for (int at = threadIdx.x; at < L * V * P && at < p.width; at += kThreads) {
        float all = part[at];
        for (int g = 1; g < kAtOnce; ++g) all += part[g * (L * V * P) + at];
        to[at] = all;
      }
    } else {
      for (int j = 0; j < P; ++j)
        for (int i = 0; i < V; ++i) {
          const int at = (j * L + lane) * V + i;
          if (at < p.width) to[at] = d[j][i];
        }
    }
  }
}

// The weights' gradients from the workgroups' parts, added in order in binary64: 6 us for 256 parts of 3 x 4096.
__global__ void __launch_bounds__(1024) k_norm_weights(NormArgs p) {
  __shared__ double sums[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, k = blockIdx.y;
  float* to = k == 0 ? p.d_post_weight : k == 1 ? p.d_scale : p.d_pre_weight;
  if (to == nullptr) return;
  const int c = blockIdx.x * 64 + lane;
  double sum = 0.0;
  const float* part = p.partial + static_cast<int64_t>(k) * p.groups * p.width + c;
  if (c < p.width)
    for (int g = w; g < p.groups; g += 128) {
      float x[8];                     // under way together
      for (int j = 0; j < 8; ++j) x[j] = g + 16 * j < p.groups ? part[static_cast<int64_t>(g + 16 * j) * p.width] : 0.0f;
      for (int j = 0; j < 8; ++j) sum += x[j];
    }
  sums[w][lane] = sum;
  __syncthreads();
  if (w != 0 || c >= p.width) return;
  for (int s = 1; s < 16; ++s) sum += sums[s][lane];
  to[c] = static_cast<float>(sum);
}

// Whether all rows lie on 16-byte boundaries and hold whole pieces.
bool in_pieces(const NormArgs& a, int esize) {
  const NormRows* all[] = {&a.block, &a.gate, &a.residual, &a.out, &a.normed, &a.d_out, &a.d_normed, &a.d_block, &a.d_gate,
                           &a.d_residual};
  if (a.width * esize % 16 != 0) return false;
  for (const NormRows* r : all)
    if (r->p && (reinterpret_cast<uintptr_t>(r->p) % 16 != 0 || r->stride * esize % 16 != 0)) return false;
  return true;
}

template <typename T, bool IN16, bool BACK>
void launch(const NormArgs& a, int dtype, hipStream_t s) {
  const NormShape n = norm_shape(a.width, dtype, BACK);
  const int64_t all = (static_cast<int64_t>(a.rows) + norm_rows_at_once(n) - 1) / norm_rows_at_once(n);
  const dim3 grid(static_cast<uint32_t>(BACK ? a.groups : all < kGrid ? all : kGrid));
  const auto go = [&](auto lanes, auto pieces) {
    constexpr int L = decltype(lanes)::value, P = decltype(pieces)::value;
    if (n.lanes != L || n.pieces != P) return;
    if constexpr (BACK) k_norm_backward<T, IN16, L, P><<<grid, threads_of(L), 0, s>>>(a);
    else k_norm<T, IN16, L, P><<<grid, threads_of(L), 0, s>>>(a);
  };
  const std::integral_constant<int, 1> one{};
  go(std::integral_constant<int, 4>{}, one);
  go(std::integral_constant<int, 16>{}, one);
  go(std::integral_constant<int, 64>{}, one);
  go(std::integral_constant<int, 128>{}, one);
  go(std::integral_constant<int, 256>{}, one);
  go(std::integral_constant<int, 512>{}, one);
  if constexpr (BACK) go(std::integral_constant<int, 512>{}, std::integral_constant<int, sizeof(T)>{});
  if constexpr (!BACK || sizeof(T) == 4) go(std::integral_constant<int, 1024>{}, one);
  if constexpr (!BACK || sizeof(T) == 2) go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
  if constexpr (sizeof(T) == 4) go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
}

template <typename T, bool BACK>
void launch(const NormArgs& a, int dtype, hipStream_t s) {
  if (in_pieces(a, sizeof(T))) launch<T, true, BACK>(a, dtype, s);
  else launch<T, false, BACK>(a, dtype, s);
}

template <bool BACK>
void launch(const NormArgs& a, int dtype, hipStream_t s) {
  if (dtype == STEPQ_BF16) launch<__bf16, BACK>(a, dtype, s);
  else if (dtype == STEPQ_F16) launch<_Float16, BACK>(a, dtype, s);
  else launch<float, BACK>(a, dtype, s);
}

}  // namespace

hipError_t launch_norm_forward(const NormArgs& a, int dtype, hipStream_t s) {
  launch<false>(a, dtype, s);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs& a, int dtype, hipStream_t s) {
  if (a.rows > 0) {
    launch<true>(a, dtype, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.d_post_weight == nullptr && a.d_scale == nullptr && a.d_pre_weight == nullptr) return hipSuccess;
  k_norm_weights<<<dim3(static_cast<uint32_t>((a.width + 63) / 64), 3), 1024, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace stepq
