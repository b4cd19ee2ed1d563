// gfx950 kernels of the gated linear recurrence: ragged prompts, their backward
// pass, and single tokens.
//
//   a_t = exp(-rate s(ga_t) softplus(decay)),  b_t = sqrt(1 - a_t^2)
//   h_t = a_t h_{t-1} + u_t,  u_t = b_t s(gx_t) x_t,  y_t = h_t
//
// A run of tokens is an affine map of the state before it, h -> A h + B, and maps
// of neighbouring runs compose.  A wave holds kScanTokens tokens of 64 V channels, the
// kScanRows waves of a workgroup follow each other in time, so each works out its map,
// the maps meet in LDS, and every wave then walks its tokens from the state that it
// starts from.
//
// Backward, with c_t = a_{t+1} g_{t+1} what comes from the tokens behind (the final
// state's gradient for the last one), g_t = dy_t + c_t:
//   dx_t = g_t b_t s(gx_t),   dgx_t = g_t u_t (1 - s(gx_t))
//   P_t = (d log a_t) log a_t = g_t (a_t h_{t-1} log a_t - a_t^2 s(gx_t) x_t log a_t / b_t)
//   dga_t = P_t (1 - s(ga_t)),   ddecay = sum_t P_t s(decay) / softplus(decay)
// c is a recurrence of the same kind, backwards: c -> a_t c + a_t dy_t.  log a / b goes to 0
// with log a, like -sqrt(-log a / 2).
#include "scan_internal.hpp"

namespace stepq {
namespace {

constexpr int R = kScanTokens;
constexpr int W = kScanRows;
constexpr int kThreads = 64 * W;
constexpr float kLog2e = 1.4426950408889634f;

// V neighbouring channels of a token.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load(const T* p) {
  return *reinterpret_cast<const Vec<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&x)[V]) {
  Vec<T, V> r;
  for (int i = 0; i < V; ++i) r.v[i] = static_cast<T>(x[i]);
  *reinterpret_cast<Vec<T, V>*>(p) = r;
}

__device__ __forceinline__ float logistic(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// 1 - exp(z) for z <= 0, good to a few 2^-24 of itself: the series up to z^7 for |z| below
// log(2) / 2 (the next term is 1.5e-8 of the sum there), beyond it the difference, which
// the rounding of exp leaves 1.4e-7 of itself at worst.
__device__ __forceinline__ float one_less_exp(float z) {
  float s = 1.0f / 5040.0f;
  s = fmaf(s, z, 1.0f / 720.0f);
  s = fmaf(s, z, 1.0f / 120.0f);
  s = fmaf(s, z, 1.0f / 24.0f);
  s = fmaf(s, z, 1.0f / 6.0f);
  s = fmaf(s, z, 0.5f);
  s = fmaf(s, z, 1.0f);
  const float far = 1.0f - __builtin_amdgcn_exp2f(z * kLog2e);
  return z > -0.34657359f ? -z * s : far;
}

// -rate softplus(decay), the logarithm of the retention at an open gate; log1p by the
// quotient that takes the rounding of 1 + e back out.
__device__ __forceinline__ float speed_of(float decay, float rate) {
  const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(decay));
  const float w = 1.0f + e;
  const float l = w == 1.0f ? e : logf(w) * (e / (w - 1.0f));
  return -rate * (fmaxf(decay, 0.0f) + l);
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

__device__ __forceinline__ Piece request_of(const ScanArgs& p, int b, int64_t piece) {
  Piece r;
  r.request = b;
  r.first = start_of(p, b);
  const int64_t end = start_of(p, b + 1);
  r.count = static_cast<int32_t>(end > r.first ? end - r.first : 0);
  r.tile = static_cast<int32_t>(piece - (r.first / kPiece + b));
  return r;
}

__device__ __forceinline__ int slot_of(const ScanArgs& p, int b) {
  if (p.slot_ids == nullptr) return -1;
  const int slot = p.slot_ids[b];
  return slot >= 0 && slot < p.num_slots ? slot : -2;     // -2: not a slot
}

// One workgroup walks a request's pieces in order, 64 V channels of it.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) k_scan(ScanArgs p) {
  __shared__ float maps[2][W][2][64 * V];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x / p.blocks, c = (blockIdx.x % p.blocks) * 64 * V + lane * V;
  const bool mine = c < p.width;
  const int cc = mine ? c : 0;
  const int64_t piece0 = start_of(p, b) / kPiece + b;
  const Piece q = request_of(p, b, piece0);
  const int slot = slot_of(p, b);
  float H[V], speed[V];
  for (int v = 0; v < V; ++v) {
    speed[v] = speed_of(p.decay[cc + v], p.rate);
    H[v] = slot >= 0 && p.resume != nullptr && p.resume[b] != 0 ? p.state[static_cast<int64_t>(slot) * p.width + cc + v] : 0.0f;
    if (slot == -2) H[v] = __builtin_nanf("");
  }
  const T* x = static_cast<const T*>(p.x) + cc;
  const T* ga = static_cast<const T*>(p.ga) + cc;
  const T* gx = static_cast<const T*>(p.gx) + cc;
  T* y = static_cast<T*>(p.y) + cc;
  for (int tile = 0; tile * kPiece < q.count; ++tile) {
    const int64_t t0 = q.first + static_cast<int64_t>(tile) * kPiece + w * R;
    const int n = max(0, min(R, q.count - tile * kPiece - w * R));
    float a[R][V], u[R][V], A[V], B[V];
    for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f;
    for (int t = 0; t < R; ++t) {
      if (t < n) {
        const Vec<T, V> xr = load<T, V>(x + (t0 + t) * p.x_stride), gr = load<T, V>(ga + (t0 + t) * p.ga_stride),
                        ir = load<T, V>(gx + (t0 + t) * p.gx_stride);
        for (int v = 0; v < V; ++v) {
          const float less = one_less_exp(speed[v] * logistic(static_cast<float>(gr.v[v])));
          a[t][v] = 1.0f - less;
          u[t][v] = __builtin_amdgcn_sqrtf(less * (1.0f + a[t][v])) * logistic(static_cast<float>(ir.v[v])) *
                    static_cast<float>(xr.v[v]);
        }
      } else {
        for (int v = 0; v < V; ++v) a[t][v] = 1.0f, u[t][v] = 0.0f;
      }
      for (int v = 0; v < V; ++v) A[v] *= a[t][v], B[v] = fmaf(a[t][v], B[v], u[t][v]);
    }
    for (int v = 0; v < V; ++v) maps[tile & 1][w][0][lane * V + v] = A[v], maps[tile & 1][w][1][lane * V + v] = B[v];
    __syncthreads();
    float h[V];
    for (int s = 0; s < W; ++s)
      for (int v = 0; v < V; ++v) {
        if (s == w) h[v] = H[v];
        H[v] = fmaf(maps[tile & 1][s][0][lane * V + v], H[v], maps[tile & 1][s][1][lane * V + v]);
      }
    if (p.saved != nullptr && mine)
      for (int v = 0; v < V; ++v) p.saved[((piece0 + tile) * W + w) * p.width + c + v] = h[v];
    for (int t = 0; t < R; ++t) {
      for (int v = 0; v < V; ++v) h[v] = fmaf(a[t][v], h[v], u[t][v]);
      if (t < n && mine) store<T, V>(y + (t0 + t) * p.y_stride, h);
    }
  }
  if (w == 0 && slot >= 0 && mine)
    for (int v = 0; v < V; ++v) p.state[static_cast<int64_t>(slot) * p.width + c + v] = H[v];
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) k_scan_backward(ScanArgs p) {
  __shared__ float maps[2][W][2][64 * V];
  __shared__ float parts[W][64 * V];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int b = blockIdx.x / p.blocks, c = (blockIdx.x % p.blocks) * 64 * V + lane * V;
  const bool mine = c < p.width;
  const int cc = mine ? c : 0;
  const int64_t piece0 = start_of(p, b) / kPiece + b;
  const Piece q = request_of(p, b, piece0);
  const int slot = slot_of(p, b);
  const int tiles = (q.count + kPiece - 1) / kPiece;
  // pieces of no tokens add nothing
  const int64_t until = b + 1 < p.batch ? start_of(p, b + 1) / kPiece + b + 1 : p.pieces;
  if (w == 0 && mine) {
    for (int64_t j = b == 0 ? 0 : piece0 + tiles; j < until; ++j)
      if (j < piece0 || j >= piece0 + tiles)
        for (int v = 0; v < V; ++v) p.partial[j * p.width + c + v] = 0.0f;
  }
  float G[V], speed[V];
  for (int v = 0; v < V; ++v) {
    speed[v] = speed_of(p.decay[cc + v], p.rate);
    G[v] = slot >= 0 ? p.state[static_cast<int64_t>(slot) * p.width + cc + v] : 0.0f;
  }
  const T* x = static_cast<const T*>(p.x) + cc;
  const T* ga = static_cast<const T*>(p.ga) + cc;
  const T* gx = static_cast<const T*>(p.gx) + cc;
  const T* dy = static_cast<const T*>(p.dy) + cc;
  T* dx = static_cast<T*>(p.y) + cc;
  T* dga = static_cast<T*>(p.dga) + cc;
  T* dgx = static_cast<T*>(p.dgx) + cc;
  for (int tile = tiles - 1; tile >= 0; --tile) {
    const int64_t t0 = q.first + static_cast<int64_t>(tile) * kPiece + w * R;
    const int n = max(0, min(R, q.count - tile * kPiece - w * R));
    float less[R][V], ra[R][V], A[V], B[V];
    Vec<T, V> gr[R];
    for (int v = 0; v < V; ++v) A[v] = 1.0f, B[v] = 0.0f;
    for (int t = R - 1; t >= 0; --t) {
      for (int v = 0; v < V; ++v) less[t][v] = 0.0f, ra[t][v] = 0.0f, gr[t].v[v] = static_cast<T>(0.0f);
      if (t < n) {
        const Vec<T, V> ar = load<T, V>(ga + (t0 + t) * p.ga_stride);
        gr[t] = load<T, V>(dy + (t0 + t) * p.dy_stride);
        for (int v = 0; v < V; ++v) {
          ra[t][v] = logistic(static_cast<float>(ar.v[v]));
          less[t][v] = one_less_exp(speed[v] * ra[t][v]);
        }
      }
      for (int v = 0; v < V; ++v) {
        const float a = 1.0f - less[t][v];
        A[v] *= a, B[v] = a * (B[v] + static_cast<float>(gr[t].v[v]));
      }
    }
    for (int v = 0; v < V; ++v) maps[tile & 1][w][0][lane * V + v] = A[v], maps[tile & 1][w][1][lane * V + v] = B[v];
    __syncthreads();
    float g[V], h[V], sum[V];
    for (int s = W - 1; s >= 0; --s)
      for (int v = 0; v < V; ++v) {
        if (s == w) g[v] = G[v];
        G[v] = fmaf(maps[tile & 1][s][0][lane * V + v], G[v], maps[tile & 1][s][1][lane * V + v]);
      }
    for (int v = 0; v < V; ++v) sum[v] = 0.0f, h[v] = p.saved[((piece0 + tile) * W + w) * p.width + cc + v];
    float before[R][V];
    Vec<T, V> xr[R], ir[R];
    for (int t = 0; t < R; ++t)
      if (t < n) {
        xr[t] = load<T, V>(x + (t0 + t) * p.x_stride), ir[t] = load<T, V>(gx + (t0 + t) * p.gx_stride);
        for (int v = 0; v < V; ++v) {
          const float a = 1.0f - less[t][v];
          before[t][v] = h[v];
          h[v] = fmaf(a, h[v], __builtin_amdgcn_sqrtf(less[t][v] * (1.0f + a)) * logistic(static_cast<float>(ir[t].v[v])) *
                                   static_cast<float>(xr[t].v[v]));
        }
      }
    for (int t = R - 1; t >= 0; --t)
      if (t < n) {
        float ox[V], oa[V], oi[V];
        for (int v = 0; v < V; ++v) {
          const float a = 1.0f - less[t][v], b2 = less[t][v] * (1.0f + a), ri = logistic(static_cast<float>(ir[t].v[v]));
          const float la = speed[v] * ra[t][v], root = __builtin_amdgcn_sqrtf(b2);
          const float slope = b2 > 0.0f ? la * __builtin_amdgcn_rcpf(root) : 0.0f;      // log a / b
          const float gain = ri * static_cast<float>(xr[t].v[v]);
          const float now = g[v] + static_cast<float>(gr[t].v[v]);
          const float P = now * a * (before[t][v] * la - a * gain * slope);
          ox[v] = now * root * ri;
          oi[v] = now * root * gain * (1.0f - ri);
          oa[v] = P * (1.0f - ra[t][v]);
          sum[v] += P;
          g[v] = a * now;
          if (slot == -2) ox[v] = oi[v] = oa[v] = __builtin_nanf(""), sum[v] = 0.0f;
        }
        if (mine) {
          store<T, V>(dx + (t0 + t) * p.y_stride, ox);
          store<T, V>(dga + (t0 + t) * p.dga_stride, oa);
          store<T, V>(dgx + (t0 + t) * p.dgx_stride, oi);
        }
      }
    for (int v = 0; v < V; ++v) parts[w][lane * V + v] = sum[v];
    __syncthreads();
    if (w == 0 && mine)
      for (int v = 0; v < V; ++v) {
        float all = 0.0f;
        for (int s = 0; s < W; ++s) all += parts[s][lane * V + v];
        p.partial[(piece0 + tile) * p.width + c + v] = all;
      }
    __syncthreads();
  }
  if (w == 0 && slot >= 0 && mine)
    for (int v = 0; v < V; ++v)
      p.state[static_cast<int64_t>(slot) * p.width + c + v] = p.resume != nullptr && p.resume[b] != 0 ? G[v] : 0.0f;
}

// ddecay from the pieces' parts, added in order in binary64: a wave takes 64 channels and
// every 16th piece.
__global__ void __launch_bounds__(1024) k_scan_decay(ScanArgs p) {
  __shared__ double sums[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  double sum = 0.0;
  if (c < p.width)
    for (int64_t j = w; j < p.pieces; j += 16) sum += p.partial[j * p.width + c];
  sums[w][lane] = sum;
  __syncthreads();
  if (w != 0 || c >= p.width) return;
  for (int s = 1; s < 16; ++s) sum += sums[s][lane];
  // s(decay) / softplus(decay) goes to 1 where both vanish
  const double e = exp(-fabs(static_cast<double>(p.decay[c]))), d = p.decay[c];
  const double soft = (d > 0.0 ? d : 0.0) + log1p(e), open = d > 0.0 ? 1.0 / (1.0 + e) : e / (1.0 + e);
  p.ddecay[c] = static_cast<float>(soft > 0.0 ? sum * (open / soft) : sum);
}

template <typename T, int V>
__global__ void __launch_bounds__(256) k_scan_step(ScanArgs p) {
  const int groups = (p.width + 256 * V - 1) / (256 * V);
  const int b = blockIdx.x / groups, c = (static_cast<int>(blockIdx.x % groups) * 256 + static_cast<int>(threadIdx.x)) * V;
  if (c >= p.width) return;
  const int slot = p.slot_ids[b];
  float h[V];
  if (slot < 0 || slot >= p.num_slots) {
    for (int v = 0; v < V; ++v) h[v] = __builtin_nanf("");
    store<T, V>(static_cast<T*>(p.y) + b * p.y_stride + c, h);
    return;
  }
  const Vec<T, V> xr = load<T, V>(static_cast<const T*>(p.x) + b * p.x_stride + c),
                  gr = load<T, V>(static_cast<const T*>(p.ga) + b * p.ga_stride + c),
                  ir = load<T, V>(static_cast<const T*>(p.gx) + b * p.gx_stride + c);
  float* at = p.state + static_cast<int64_t>(slot) * p.width + c;
  for (int v = 0; v < V; ++v) {
    const float less = one_less_exp(speed_of(p.decay[c + v], p.rate) * logistic(static_cast<float>(gr.v[v])));
    const float a = 1.0f - less;
    h[v] = fmaf(a, at[v], __builtin_amdgcn_sqrtf(less * (1.0f + a)) * logistic(static_cast<float>(ir.v[v])) *
                              static_cast<float>(xr.v[v]));
    at[v] = h[v];
  }
  store<T, V>(static_cast<T*>(p.y) + b * p.y_stride + c, h);
}

// Two channels a lane where every pair lies on a boundary of its size.
bool in_pairs(const ScanArgs& a, int esize) {
  const auto pair = [&](const void* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % (2 * esize) == 0 && stride % 2 == 0;
  };
  return a.width % 2 == 0 && pair(a.x, a.x_stride) && pair(a.ga, a.ga_stride) && pair(a.gx, a.gx_stride) &&
         pair(a.y, a.y_stride) && pair(a.dy, a.dy_stride) && pair(a.dga, a.dga_stride) && pair(a.dgx, a.dgx_stride);
}

template <typename T>
hipError_t forward(ScanArgs a, hipStream_t s) {
  const bool two = in_pairs(a, sizeof(T));
  a.blocks = two ? (a.width + 127) / 128 : (a.width + 63) / 64;
  const dim3 grid(static_cast<uint32_t>(static_cast<int64_t>(a.batch) * a.blocks));
  if (two) k_scan<T, 2><<<grid, kThreads, 0, s>>>(a);
  else k_scan<T, 1><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t backward(ScanArgs a, hipStream_t s) {
  if (a.pieces > 0) {
    const bool two = in_pairs(a, sizeof(T));
    a.blocks = two ? (a.width + 127) / 128 : (a.width + 63) / 64;
    const dim3 grid(static_cast<uint32_t>(static_cast<int64_t>(a.batch) * a.blocks));
    if (two) k_scan_backward<T, 2><<<grid, kThreads, 0, s>>>(a);
    else k_scan_backward<T, 1><<<grid, kThreads, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  k_scan_decay<<<dim3(static_cast<uint32_t>((a.width + 63) / 64)), 1024, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t step(const ScanArgs& a, hipStream_t s) {
  const bool two = in_pairs(a, sizeof(T));
  const int channels = two ? 512 : 256;
  const dim3 grid(static_cast<uint32_t>(static_cast<int64_t>(a.batch) * ((a.width + channels - 1) / channels)));
  if (two) k_scan_step<T, 2><<<grid, 256, 0, s>>>(a);
  else k_scan_step<T, 1><<<grid, 256, 0, s>>>(a);
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
