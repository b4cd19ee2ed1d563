// gfx950 kernels of linear attention with one decay per head: ragged prompts
// in chunks of 64 tokens, and single tokens.
//
// State of a (request, value head): M [D key channels][D value channels].
//   additive rule  M_t = a_t M_{t-1} + k_t v_t^T
//   delta rule     M_t = a_t M_{t-1} + b_t k_t (v_t - a_t M_{t-1}^T k_t)^T
//   o_t = M_t^T q_t
//
// Chunked form.  With G_t the product of the chunk's retentions up to token t
// and M the state before the chunk, M_t = G_t M + sum_{j <= t} (G_t / G_j) k_j
// u_j^T where u_j = v_j (additive), or (delta)
//   u_t = b_t (v_t - G_t M^T k_t - sum_{j < t} (G_t / G_j) (k_j . k_t) u_j),
// that is (I + B) U = diag(b) (V - diag(G) K M) with the strictly lower
// triangular B_tj = b_t (G_t / G_j) k_t . k_j.  So, per chunk,
//   U = T (V - diag(G) K M),  T = (I + B)^-1 diag(b)
//   O = diag(G) Q M + A U,    A_tj = (G_t / G_j) q_t . k_j  for j <= t
//   M <- G_C M + K^T diag(G_C / G) U
// T and A do not depend on the state: k_linear_chunks computes them for all
// chunks at once.  k_linear_walk then walks a request's chunks in order; value
// columns are independent there, so a workgroup owns some columns of one head.
#include "linear_internal.hpp"

namespace stepq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16;
typedef _Float16 f16;
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

constexpr int C = kChunk;
constexpr int kThreads = 256;

// Eight consecutive elements of a 16-byte aligned row, as floats.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
  for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
}
__device__ __forceinline__ void load8(const bf16* p, float (&x)[8]) {
  const u16x8 a = *reinterpret_cast<const u16x8*>(p);
  for (int i = 0; i < 8; ++i) x[i] = __builtin_bit_cast(float, static_cast<uint32_t>(a[i]) << 16);
}
__device__ __forceinline__ void load8(const f16* p, float (&x)[8]) {
  const u16x8 a = *reinterpret_cast<const u16x8*>(p);
  for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(__builtin_bit_cast(f16, static_cast<uint16_t>(a[i])));
}

// Product of a 16 x 32 and a 32 x 16 block in binary32.  A lane's eight values
// of either operand belong to depth 4 g + j (j < 4) and 16 + 4 g + j - 4, with
// g = lane / 16: in this order the two accumulator tiles that make up 32 rows
// of a product are the next product's operand as they stand.
struct Frag {
  float v[8];
};
__device__ __forceinline__ Frag from_tiles(const f32x4& lo, const f32x4& hi) {
  Frag f;
  for (int j = 0; j < 4; ++j) f.v[j] = lo[j], f.v[4 + j] = hi[j];
  return f;
}
__device__ __forceinline__ f32x4 mma(const Frag& a, const Frag& b, f32x4 c) {
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], c, 0, 0, 0);
  return c;
}
__device__ __forceinline__ f32x4 mma16(const f32x4& a, const f32x4& b, f32x4 c) {   // 16 deep
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
  return c;
}
// Operand with rows along the row axis of x (row-major, stride ld): row = lane % 16.
__device__ __forceinline__ Frag rows_of(const float* x, int ld, int lane) {
  const float* p = x + (lane & 15) * ld + 4 * (lane >> 4);
  return from_tiles(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 16));
}
// Operand with rows along the column axis of x: row = column lane % 16 of x.
__device__ __forceinline__ Frag cols_of(const float* x, int ld, int lane) {
  const float* p = x + 4 * (lane >> 4) * ld + (lane & 15);
  Frag f;
  for (int j = 0; j < 4; ++j) f.v[j] = p[j * ld], f.v[4 + j] = p[(16 + j) * ld];
  return f;
}

template <int D>
struct Dims {
  static constexpr int DP = D < 32 ? 32 : D;   // depth of products over key channels, zero-padded to 32
  static constexpr int LD = DP + 4;            // row stride in LDS (bank spread)
  static constexpr int KB = DP / 32;
  static constexpr int RT = D / 16;
};

struct Span {
  int64_t first;   // token index of the chunk's or request's first row
  int32_t count;
};

__device__ __forceinline__ Span request_span(const LinearArgs& a, int b) {
  const int64_t n = a.total_tokens;
  int64_t lo = a.cu_seqlens[b], hi = a.cu_seqlens[b + 1];
  lo = lo < 0 ? 0 : (lo > n ? n : lo);
  hi = hi < lo ? lo : (hi > n ? n : hi);
  return {lo, static_cast<int32_t>(hi - lo)};
}

// One (chunk, head) of the workspace: T and A (row-major C x C), then the
// retentions G_t and G_C / G_t.
struct ChunkWs {
  float* t;
  float* a;
  float* grow;
  float* left;
};
__device__ __forceinline__ ChunkWs chunk_ws(uint8_t* ws, int64_t index, bool delta) {
  float* p = reinterpret_cast<float*>(ws) + index * ((delta ? 2 : 1) * C * C + 2 * C);
  ChunkWs w;
  w.grow = p;
  w.left = p + C;
  w.a = p + 2 * C;
  w.t = delta ? w.a + C * C : nullptr;
  return w;
}

// Rows first .. first+C-1 of a head of q or k into LDS as floats, zeros past
// `count` tokens and past D channels.
template <int D, typename T>
__device__ __forceinline__ void stage(float* lds, const T* x, int64_t stride, int count) {
  constexpr int DP = Dims<D>::DP, LD = Dims<D>::LD, PR = DP / 8;
  for (int i = threadIdx.x; i < C * PR; i += blockDim.x) {
    const int row = i / PR, col = (i % PR) * 8;
    float x8[8] = {};
    if (row < count && col < D) load8(x + row * stride + col, x8);
    float* p = lds + row * LD + col;
    *reinterpret_cast<f32x4*>(p) = f32x4{x8[0], x8[1], x8[2], x8[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{x8[4], x8[5], x8[6], x8[7]};
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) k_linear_chunks(LinearArgs p) {
  using S = Dims<D>;
  constexpr int LS = C + 4;
  __shared__ __align__(16) float kq[2][C * S::LD];
  __shared__ __align__(16) float low[C * LS];
  __shared__ __align__(16) float inv[4][16 * 20];
  __shared__ double lg[C];
  __shared__ float bt[C];
  const bool delta = p.beta != nullptr;
  const int h = blockIdx.x % p.H;
  const int64_t w = blockIdx.x / p.H;
  // the request whose range of chunk indices holds w: the last b with cu[b] / C + b <= w
  int b = 0;
  for (int lo = 0, hi = p.batch - 1; lo <= hi;) {
    const int mid = (lo + hi) / 2;
    if (request_span(p, mid).first / C + mid <= w) b = mid, lo = mid + 1;
    else hi = mid - 1;
  }
  const Span r = request_span(p, b);
  const int64_t c = w - (r.first / C + b);
  if (c < 0 || c * C >= r.count) return;
  const int64_t first = r.first + c * C;
  const int count = min(C, static_cast<int>(r.count - c * C));
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4;

  stage<D>(kq[0], static_cast<const T*>(p.k) + first * p.k_stride + (h / p.rep) * D, p.k_stride, count);
  stage<D>(kq[1], static_cast<const T*>(p.q) + first * p.q_stride + (h / p.rep) * D, p.q_stride, count);
  const ChunkWs ws = chunk_ws(p.workspace, w * p.H + h, delta);
  if (wave == 0) {
    // log2 G as a running sum in binary64, so that ratios of retentions far
    // into a fast-forgetting chunk keep binary32 accuracy; a retention of 0 (or
    // below 2^-200) counts as 2^-200, which leaves nothing in binary32
    double x = 0.0;
    if (lane < count) {
      x = log2(static_cast<double>(p.gate[(first + lane) * p.H + h]));
      if (x < -200.0) x = -200.0;
    }
    for (int s = 1; s < 64; s <<= 1) {
      const double y = __shfl_up(x, s);
      if (lane >= s) x += y;
    }
    const double all = __shfl(x, 63);
    lg[lane] = x;
    bt[lane] = delta && lane < count ? p.beta[(first + lane) * p.H + h] : 0.0f;
    ws.grow[lane] = exp2f(static_cast<float>(x));
    ws.left[lane] = exp2f(static_cast<float>(all - x));
  }
  __syncthreads();

  // rows 16 wave .. 16 wave + 15 of K K^T and Q K^T
  for (int ct = 0; ct < 4; ++ct) {
    f32x4 kk = {}, qk = {};
    if (ct <= wave)
      for (int kb = 0; kb < S::KB; ++kb) {
        const Frag kr = rows_of(kq[0] + 16 * ct * S::LD + 32 * kb, S::LD, lane);
        if (delta) kk = mma(rows_of(kq[0] + 16 * wave * S::LD + 32 * kb, S::LD, lane), kr, kk);
        qk = mma(rows_of(kq[1] + 16 * wave * S::LD + 32 * kb, S::LD, lane), kr, qk);
      }
    const int j = 16 * ct + (lane & 15);
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * wave + 4 * g + e;
      const float ratio = exp2f(static_cast<float>(lg[i] - lg[j]));
      ws.a[i * C + j] = j <= i ? qk[e] * ratio : 0.0f;
      if (delta) low[i * LS + j] = j < i ? kk[e] * ratio * bt[i] : 0.0f;
    }
  }
  if (!delta) return;
  __syncthreads();

  // (I + B)^-1.  Diagonal blocks of 16 by forward substitution, one column per
  // lane; the rest by blocks, T_ij = -T_ii sum_k B_ik T_kj, wave j doing block
  // column j: both are as stable as the substitution that defines U.
  if (wave == 0) {
    const float* lb = low + (16 * g) * LS + 16 * g;
    float x[16];
    for (int i = 0; i < 16; ++i) {
      float s = i == (lane & 15) ? 1.0f : 0.0f;
      for (int j = 0; j < i; ++j) s = fmaf(-lb[i * LS + j], x[j], s);
      x[i] = s;
    }
    for (int i = 0; i < 16; ++i) inv[g][i * 20 + (lane & 15)] = x[i];
  }
  __syncthreads();
  f32x4 col[4];
  const int j = 16 * wave + (lane & 15);
  for (int i = 0; i < 4; ++i) {
    if (i < wave) {
      col[i] = f32x4{};
    } else if (i == wave) {
      for (int e = 0; e < 4; ++e) col[i][e] = inv[i][(4 * g + e) * 20 + (lane & 15)];
    } else {
      f32x4 s = {};
      for (int k = 0; k < i; ++k)
        if (k >= wave)
          s = mma16(*reinterpret_cast<const f32x4*>(low + (16 * i + (lane & 15)) * LS + 16 * k + 4 * g), col[k], s);
      f32x4 ti = *reinterpret_cast<const f32x4*>(&inv[i][(lane & 15) * 20 + 4 * g]);
      col[i] = mma16(-ti, s, f32x4{});
    }
    for (int e = 0; e < 4; ++e) ws.t[(16 * i + 4 * g + e) * C + j] = col[i][e] * bt[j];
  }
}

template <int D, typename T, int NW>
__global__ void __launch_bounds__(64 * NW) k_linear_walk(LinearArgs p) {
  using S = Dims<D>;
  constexpr int LA = C + 4;
  constexpr int SPLIT = D / (16 * NW);   // workgroups per head
  extern __shared__ __align__(16) float lds[];
  float* lk = lds;
  float* lq = lk + C * S::LD;
  float* la = lq + C * S::LD;
  float* lt = la + C * LA;
  __shared__ float grow[C], left[C];
  const bool delta = p.beta != nullptr;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4;
  const int h = (blockIdx.x / SPLIT) % p.H;
  const int b = blockIdx.x / (SPLIT * p.H);
  const int vcol = (blockIdx.x % SPLIT) * 16 * NW + 16 * wave + (lane & 15);
  const Span r = request_span(p, b);
  const int slot = p.slot_ids[b];
  T* o = static_cast<T*>(p.o) + r.first * p.o_stride + h * D + vcol;
  if (slot < 0 || slot >= p.num_slots) {
    for (int t = g; t < r.count; t += 4) o[t * p.o_stride] = static_cast<T>(__builtin_nanf(""));
    return;
  }
  const T* v = static_cast<const T*>(p.v) + r.first * p.v_stride + h * D + vcol;
  const T* k = static_cast<const T*>(p.k) + r.first * p.k_stride + (h / p.rep) * D;
  const T* q = static_cast<const T*>(p.q) + r.first * p.q_stride + (h / p.rep) * D;
  float* state = p.state + (static_cast<int64_t>(slot) * p.H + h) * D * D + vcol;

  f32x4 m[S::RT];   // column vcol; tile i holds key channels 16 i + 4 g + e
  const bool go_on = p.resume != nullptr && p.resume[b] != 0;
  for (int i = 0; i < S::RT; ++i)
    for (int e = 0; e < 4; ++e) m[i][e] = go_on ? state[(16 * i + 4 * g + e) * D] : 0.0f;

  const int64_t base = r.first / C + b;
  for (int c = 0; c * C < r.count; ++c) {
    const int count = min(C, r.count - c * C);
    const int64_t t0 = static_cast<int64_t>(c) * C;
    const ChunkWs ws = chunk_ws(p.workspace, (base + c) * p.H + h, delta);
    __syncthreads();
    stage<D>(lk, k + t0 * p.k_stride, p.k_stride, count);
    stage<D>(lq, q + t0 * p.q_stride, p.q_stride, count);
    for (int i = tid; i < C * C / 4; i += 64 * NW) {
      const int row = i / (C / 4), col = i % (C / 4) * 4;
      *reinterpret_cast<f32x4*>(la + row * LA + col) = reinterpret_cast<const f32x4*>(ws.a)[i];
      if (delta) *reinterpret_cast<f32x4*>(lt + row * LA + col) = reinterpret_cast<const f32x4*>(ws.t)[i];
    }
    for (int i = tid; i < C; i += 64 * NW) grow[i] = ws.grow[i], left[i] = ws.left[i];
    f32x4 u[4];
    for (int i = 0; i < 4; ++i)
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * i + 4 * g + e;
        u[i][e] = t < count ? static_cast<float>(v[(t0 + t) * p.v_stride]) : 0.0f;
      }
    __syncthreads();

    Frag mf[S::KB];
    for (int kb = 0; kb < S::KB; ++kb) mf[kb] = from_tiles(m[2 * kb], D < 32 ? f32x4{} : m[D < 32 ? 0 : 2 * kb + 1]);
    if (delta) {
      for (int i = 0; i < 4; ++i) {
        f32x4 s = {};
        for (int kb = 0; kb < S::KB; ++kb) s = mma(rows_of(lk + 16 * i * S::LD + 32 * kb, S::LD, lane), mf[kb], s);
        for (int e = 0; e < 4; ++e) u[i][e] -= grow[16 * i + 4 * g + e] * s[e];
      }
      const Frag rf[2] = {from_tiles(u[0], u[1]), from_tiles(u[2], u[3])};
      for (int i = 0; i < 4; ++i) {
        f32x4 s = mma(rows_of(lt + 16 * i * LA, LA, lane), rf[0], f32x4{});
        if (i >= 2) s = mma(rows_of(lt + 16 * i * LA + 32, LA, lane), rf[1], s);
        u[i] = s;
      }
    }
    const Frag uf[2] = {from_tiles(u[0], u[1]), from_tiles(u[2], u[3])};
    for (int i = 0; i < 4; ++i) {
      f32x4 s = {};
      for (int kb = 0; kb < S::KB; ++kb) s = mma(rows_of(lq + 16 * i * S::LD + 32 * kb, S::LD, lane), mf[kb], s);
      for (int e = 0; e < 4; ++e) s[e] *= grow[16 * i + 4 * g + e];
      s = mma(rows_of(la + 16 * i * LA, LA, lane), uf[0], s);
      if (i >= 2) s = mma(rows_of(la + 16 * i * LA + 32, LA, lane), uf[1], s);
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * i + 4 * g + e;
        if (t < count) o[(t0 + t) * p.o_stride] = static_cast<T>(s[e]);
      }
    }
    for (int i = 0; i < 4; ++i)
      for (int e = 0; e < 4; ++e) u[i][e] *= left[16 * i + 4 * g + e];
    const Frag wf[2] = {from_tiles(u[0], u[1]), from_tiles(u[2], u[3])};
    const float all = grow[C - 1];
    for (int i = 0; i < S::RT; ++i) {
      f32x4 s = m[i] * all;
      for (int tb = 0; tb < 2; ++tb) s = mma(cols_of(lk + 32 * tb * S::LD + 16 * i, S::LD, lane), wf[tb], s);
      m[i] = s;
    }
  }
  for (int i = 0; i < S::RT; ++i)
    for (int e = 0; e < 4; ++e) state[(16 * i + 4 * g + e) * D] = m[i][e];
}

// One token: a workgroup owns CW columns of one (request, head) state; a lane
// holds 4 columns of D / RG rows in registers.  With the decayed state M~,
// u = M~^T k and w = M~^T q (one reduction for both) the new state's readout is
// o = w + (q . k) x with x = b (v - u), or v for the additive rule, so the state
// is read and written once.
template <int D, typename T, int CW>
__global__ void __launch_bounds__(kThreads) k_linear_step(LinearArgs p) {
  constexpr int LPR = CW / 4;
  constexpr int NT = D * LPR < kThreads ? (D * LPR < 64 ? 64 : D * LPR) : kThreads;
  constexpr int RG = NT / LPR;                 // row groups
  constexpr int RPT = (D + RG - 1) / RG;       // rows per lane; row groups past D idle
  constexpr int NW = NT / 64;
  constexpr int SPLIT = D / CW;
  __shared__ float qs[D], ks[D];
  __shared__ __align__(16) f32x4 part[NW][2][LPR < 64 ? LPR : 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = (blockIdx.x / SPLIT) % p.H;
  const int64_t b = blockIdx.x / (SPLIT * p.H);
  const int j0 = (blockIdx.x % SPLIT) * CW + 4 * (tid % LPR);
  const int rg = tid / LPR;
  const int slot = p.slot_ids[b];
  T* o = static_cast<T*>(p.o) + b * p.o_stride + h * D + j0;
  if (slot < 0 || slot >= p.num_slots) {
    if (tid < LPR)
      for (int e = 0; e < 4; ++e) o[e] = static_cast<T>(__builtin_nanf(""));
    return;
  }
  float* state = p.state + (static_cast<int64_t>(slot) * p.H + h) * D * D + j0;
  f32x4 m[RPT];
  for (int i = 0; i < RPT; ++i)
    if (rg + i * RG < D) m[i] = *reinterpret_cast<const f32x4*>(state + (rg + i * RG) * D);
  if (tid < D) {
    qs[tid] = static_cast<float>(static_cast<const T*>(p.q)[b * p.q_stride + (h / p.rep) * D + tid]);
    ks[tid] = static_cast<float>(static_cast<const T*>(p.k)[b * p.k_stride + (h / p.rep) * D + tid]);
  }
  const float a = p.gate[b * p.H + h];
  const float beta = p.beta ? p.beta[b * p.H + h] : 0.0f;
  f32x4 v;
  for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(static_cast<const T*>(p.v)[b * p.v_stride + h * D + j0 + e]);
  __syncthreads();
  f32x4 u = {}, w = {};
  for (int i = 0; i < RPT; ++i)
    if (rg + i * RG < D) {
      m[i] *= a;
      u += m[i] * ks[rg + i * RG];
      w += m[i] * qs[rg + i * RG];
    }
  float qk = 0.0f;
  for (int i = lane; i < D; i += 64) qk = fmaf(qs[i], ks[i], qk);
  for (int s = 1; s < 64; s <<= 1) qk += __shfl_xor(qk, s);
  for (int s = LPR; s < 64; s <<= 1)
    for (int e = 0; e < 4; ++e) {
      u[e] += __shfl_xor(u[e], s);
      w[e] += __shfl_xor(w[e], s);
    }
  if constexpr (NW > 1) {
    if (lane < LPR) part[wave][0][lane] = u, part[wave][1][lane] = w;
    __syncthreads();
    u = w = f32x4{};
    for (int n = 0; n < NW; ++n) {
      u += part[n][0][tid % LPR];
      w += part[n][1][tid % LPR];
    }
  }
  const f32x4 x = p.beta ? beta * (v - u) : v;
  for (int i = 0; i < RPT; ++i)
    if (rg + i * RG < D) *reinterpret_cast<f32x4*>(state + (rg + i * RG) * D) = m[i] + ks[rg + i * RG] * x;
  if (tid < LPR)
    for (int e = 0; e < 4; ++e) o[e] = static_cast<T>(w[e] + qk * x[e]);
}

template <int D, typename T>
hipError_t prefill_dt(const LinearArgs& a, hipStream_t s) {
  using S = Dims<D>;
  constexpr int NW = D >= 64 ? 4 : D / 16;
  const int64_t chunks = max_chunks(a.total_tokens, a.batch);
  k_linear_chunks<D, T><<<dim3(static_cast<uint32_t>(chunks * a.H)), kThreads, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t lds = sizeof(float) * (2 * C * S::LD + (a.beta ? 2 : 1) * C * (C + 4));
  auto* kern = k_linear_walk<D, T, NW>;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                          static_cast<int>(lds));
  if (e != hipSuccess) return e;
  kern<<<dim3(static_cast<uint32_t>(a.batch * a.H * (D / (16 * NW)))), 64 * NW, lds, s>>>(a);
  return hipGetLastError();
}

template <int D, typename T>
hipError_t step_dt(const LinearArgs& a, hipStream_t s) {
  constexpr int CW = D;
  constexpr int LPR = CW / 4;
  constexpr int NT = D * LPR < kThreads ? (D * LPR < 64 ? 64 : D * LPR) : kThreads;
  k_linear_step<D, T, CW><<<dim3(static_cast<uint32_t>(a.batch * a.H * (D / CW))), NT, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t prefill_t(int d, const LinearArgs& a, hipStream_t s) {
  switch (d) {
    case 16: return prefill_dt<16, T>(a, s);
    case 32: return prefill_dt<32, T>(a, s);
    case 64: return prefill_dt<64, T>(a, s);
    default: return prefill_dt<128, T>(a, s);
  }
}
template <typename T>
hipError_t step_t(int d, const LinearArgs& a, hipStream_t s) {
  switch (d) {
    case 16: return step_dt<16, T>(a, s);
    case 32: return step_dt<32, T>(a, s);
    case 64: return step_dt<64, T>(a, s);
    default: return step_dt<128, T>(a, s);
  }
}

}  // namespace

size_t chunk_bytes(int rule, int dtype) {
  (void)dtype;
  return sizeof(float) * ((rule == STEPQ_RULE_DELTA ? 2 : 1) * C * C + 2 * C);
}

hipError_t launch_linear_prefill(const stepq_linear_desc& d, const LinearArgs& a, hipStream_t s) {
  switch (d.dtype) {
    case STEPQ_BF16: return prefill_t<bf16>(d.d, a, s);
    case STEPQ_F16: return prefill_t<f16>(d.d, a, s);
    default: return prefill_t<float>(d.d, a, s);
  }
}

hipError_t launch_linear_step(const stepq_linear_desc& d, const LinearArgs& a, hipStream_t s) {
  switch (d.dtype) {
    case STEPQ_BF16: return step_t<bf16>(d.d, a, s);
    case STEPQ_F16: return step_t<f16>(d.d, a, s);
    default: return step_t<float>(d.d, a, s);
  }
}

}  // namespace stepq
