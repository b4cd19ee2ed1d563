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
//   U = (I + B)^-1 diag(b) (V - diag(G) K M)
//   O = diag(G) Q M + A U,    A_tj = (G_t / G_j) q_t . k_j  for j <= t
//   M <- G_C M + K^T diag(G_C / G) U
// A and B do not depend on the state, and value columns are independent of each
// other.  So a request's chunks are walked in order by workgroups that own some
// columns of one head, either with A and B from a kernel that computes them for all
// chunks at once (few heads: many workgroups a head), or computing them as they go
// (no 37 KB of them a chunk and head through memory).  512 pairs of 1024 tokens,
// delta rule, bfloat16, D = 128: 408 us the first way and 273 us the second; where the
// one takes over from the other stands, with figures, in linear_internal.hpp.
//
// Binary32 inputs run on binary32 matrix instructions (k_linear_chunks,
// k_linear_walk), 16-bit inputs on bfloat16 ones (k_linear16_*).  MI355X copies at
// 5160 GB/s and multiplies large matrices at 1226 (bfloat16) and 153 (binary32)
// TFLOP/s; what each kernel reaches stands beside it.
#include "linear_internal.hpp"

namespace stepq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16;
typedef _Float16 f16;

constexpr int C = kChunk;
constexpr int kThreads = 256;

// Eight consecutive elements of a 16-byte aligned row.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
  for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
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

// Keeps the compiler from moving loads across: registers are what bounds it.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// Stands between matrix instructions and a branch.  A matrix instruction's result
// may be read only some cycles later (up to 11 wait states here), which the compiler
// sees to within a straight run of code; over a branch it has been seen to read
// too early, so no such result is left open at one.
__device__ __forceinline__ void settle() {
  in_order();
  asm volatile("s_nop 15");
  in_order();
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

// The request whose range of indices of `tokens`-token pieces holds w: the last b with
// cu_seqlens[b] / tokens + b <= w.
__device__ __forceinline__ int owner(const LinearArgs& p, int64_t w, int tokens) {
  int b = 0;
  for (int lo = 0, hi = p.batch - 1; lo <= hi;) {
    const int mid = (lo + hi) / 2;
    if (request_span(p, mid).first / tokens + mid <= w) b = mid, lo = mid + 1;
    else hi = mid - 1;
  }
  return b;
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
template <int D, typename T, int THREADS>
__device__ __forceinline__ void stage(float* lds, const T* x, int64_t stride, int count) {
  constexpr int DP = Dims<D>::DP, LD = Dims<D>::LD, PR = DP / 8, N = C * PR / THREADS;
  constexpr int AHEAD = N < 4 ? N : 4;      // loads under way at once
  for (int first = 0; first < N; first += AHEAD) {
    float x8[AHEAD][8];
    for (int j = 0; j < AHEAD; ++j) {
      const int i = threadIdx.x + (first + j) * THREADS, row = min(i / PR, count - 1), col = min(i % PR * 8, D - 8);
      load8(x + row * stride + col, x8[j]);
    }
    for (int j = 0; j < AHEAD; ++j) {
      const int i = threadIdx.x + (first + j) * THREADS, row = i / PR, col = i % PR * 8;
      const bool real = row < count && col < D;
      float* p = lds + row * LD + col;
      for (int e = 0; e < 8; e += 4) {
        const f32x4 y = {x8[j][e], x8[j][e + 1], x8[j][e + 2], x8[j][e + 3]};
        *reinterpret_cast<f32x4*>(p + e) = real ? y : f32x4{};
      }
    }
  }
}

// Block column J of (I + B)^-1 diag(beta), one wave.
template <int J>
__device__ __forceinline__ void invert_column(const float* low, int ls, const float (*inv)[16 * 20], const float* bt,
                                              float* t, int lane) {
  const int g = lane >> 4, c = lane & 15;
  f32x4 col[4] = {};
  for (int e = 0; e < 4; ++e) col[J][e] = inv[J][(4 * g + e) * 20 + c];
  for (int i = J + 1; i < 4; ++i) {
    f32x4 s = {};
    for (int k = J; k < i; ++k) s = mma16(*reinterpret_cast<const f32x4*>(low + (16 * i + c) * ls + 16 * k + 4 * g), col[k], s);
    const f32x4 ti = *reinterpret_cast<const f32x4*>(&inv[i][c * 20 + 4 * g]);
    col[i] = mma16(-ti, s, f32x4{});
  }
  settle();
  for (int i = 0; i < 4; ++i)
    for (int e = 0; e < 4; ++e) t[(16 * i + 4 * g + e) * C + 16 * J + c] = col[i][e] * bt[16 * J + c];
}

template <int D, typename T, bool DELTA>
__global__ void __launch_bounds__(kThreads) k_linear_chunks(LinearArgs p) {
  using S = Dims<D>;
  constexpr int LS = C + 4;
  __shared__ __align__(16) float kq[2][C * S::LD];
  __shared__ __align__(16) float low[C * LS];
  __shared__ __align__(16) float inv[4][16 * 20];
  __shared__ double lg[C];
  __shared__ float bt[C];
  const int h = blockIdx.x % p.H;
  const int64_t w = blockIdx.x / p.H;
  const int b = owner(p, w, C);
  const Span r = request_span(p, b);
  const int64_t c = w - (r.first / C + b);
  if (c < 0 || c * C >= r.count) return;
  const int64_t first = r.first + c * C;
  const int count = min(C, static_cast<int>(r.count - c * C));
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4;

  stage<D, T, kThreads>(kq[0], static_cast<const T*>(p.k) + first * p.k_stride + (h / p.rep) * D, p.k_stride, count);
  stage<D, T, kThreads>(kq[1], static_cast<const T*>(p.q) + first * p.q_stride + (h / p.rep) * D, p.q_stride, count);
  const ChunkWs ws = chunk_ws(p.workspace, w * p.H + h, DELTA);
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
    bt[lane] = DELTA && lane < count ? p.beta[(first + lane) * p.H + h] : 0.0f;
    ws.grow[lane] = exp2f(static_cast<float>(x));
    ws.left[lane] = exp2f(static_cast<float>(all - x));
  }
  __syncthreads();

  // rows 16 wave .. 16 wave + 15 of K K^T and Q K^T
  for (int ct = 0; ct < 4; ++ct) {
    f32x4 kk = {}, qk = {};
    for (int kb = 0; kb < S::KB; ++kb) {
      const Frag kr = rows_of(kq[0] + 16 * ct * S::LD + 32 * kb, S::LD, lane);
      if constexpr (DELTA) kk = mma(rows_of(kq[0] + 16 * wave * S::LD + 32 * kb, S::LD, lane), kr, kk);
      qk = mma(rows_of(kq[1] + 16 * wave * S::LD + 32 * kb, S::LD, lane), kr, qk);
    }
    settle();
    const int j = 16 * ct + (lane & 15);
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * wave + 4 * g + e;
      const float ratio = j <= i ? exp2f(static_cast<float>(lg[i] - lg[j])) : 0.0f;
      ws.a[i * C + j] = qk[e] * ratio;
      if constexpr (DELTA) low[i * LS + j] = j < i ? kk[e] * ratio * bt[i] : 0.0f;
    }
  }
  if constexpr (!DELTA) return;
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
  switch (wave) {
    case 0: return invert_column<0>(low, LS, inv, bt, ws.t, lane);
    case 1: return invert_column<1>(low, LS, inv, bt, ws.t, lane);
    case 2: return invert_column<2>(low, LS, inv, bt, ws.t, lane);
    default: return invert_column<3>(low, LS, inv, bt, ws.t, lane);
  }
}

// A workgroup of up to four waves for 64 columns of a head.  Bound by the latency of a
// chunk's chain of staging and dependent products: 3001 tokens of 5 requests, 12 heads
// of 64, 134 us in all, some 6 us a chunk of the longest; one wave for 16 columns
// instead, in four times as many workgroups, 172 against 131 us for this kernel.
template <int D, typename T, bool DELTA, int NW>
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
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4;
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
    const ChunkWs ws = chunk_ws(p.workspace, (base + c) * p.H + h, DELTA);
    __syncthreads();
    stage<D, T, 64 * NW>(lk, k + t0 * p.k_stride, p.k_stride, count);
    stage<D, T, 64 * NW>(lq, q + t0 * p.q_stride, p.q_stride, count);
    constexpr int N = C * C / 4 / (64 * NW), AHEAD = N < 4 ? N : 4;
    for (int first = 0; first < N; first += AHEAD) {
      f32x4 xa[AHEAD], xt[AHEAD];
      for (int j = 0; j < AHEAD; ++j) {
        const int i = tid + (first + j) * 64 * NW;
        xa[j] = reinterpret_cast<const f32x4*>(ws.a)[i];
        if constexpr (DELTA) xt[j] = reinterpret_cast<const f32x4*>(ws.t)[i];
      }
      for (int j = 0; j < AHEAD; ++j) {
        const int i = tid + (first + j) * 64 * NW, to = i / (C / 4) * LA + i % (C / 4) * 4;
        *reinterpret_cast<f32x4*>(la + to) = xa[j];
        if constexpr (DELTA) *reinterpret_cast<f32x4*>(lt + to) = xt[j];
      }
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
    if constexpr (DELTA) {
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
      settle();
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
    settle();
  }
  for (int i = 0; i < S::RT; ++i)
    for (int e = 0; e < 4; ++e) state[(16 * i + 4 * g + e) * D] = m[i][e];
}

// ------------------------------------------------ 16-bit inputs: bfloat16 parts
//
// Matrix products of 16-bit inputs run on bfloat16 matrix instructions, which
// multiply exactly and add in binary32, sixteen times as fast as the binary32
// ones.  A bfloat16 q, k or v is its own operand; a binary16 one is the sum of
// two bfloat16 parts exactly (11 bits in 8 + 8).  Computed operands (state, A, the
// system for U, U, what is added to the state) are binary32 values, the sum of
// three parts exactly (24 bits in 8 + 8 + 8), and of a product of two such operands
// the terms from 2^-24 on are left out: products are as good as binary32 ones.
// (Two parts, 2^-18.7 of the value on the average, took 0.80 to 0.98 of the time and
// left states of the delta rule 3e-6 to 5e-6 off in the 2-norm.)
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// x, in a register whose value the compiler does not know: addresses derived from
// it are computed where they are used instead of being kept through the loop over
// chunks (some 80 registers of them).
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// LDS accesses of one wave's lanes to each other's words: ordered in hardware, this
// keeps the compiler to it.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int NP>
struct Parts {
  bf16x8 p[NP];
};

__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ bf16x4 rounded(const f32x4& x) { return __builtin_convertvector(x, bf16x4); }
__device__ __forceinline__ f32x4 widened(const bf16x4& x) { return __builtin_convertvector(x, f32x4); }

// x - hi, where hi is x rounded: a dot product of a pair of hi with (-1, 0) or (0, -1)
// takes one instruction a value, with no unpacking.  All of its terms are exact.
// The factors are kept in registers: as an operand of this instruction the constant
// -1.0 does not mean the pair (-1, 0) that the compiler writes it for.
__device__ __forceinline__ f32x4 rest_of(const f32x4& x, const bf16x4& hi) {
  typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
  uint32_t f = 0x0000bf80u, s = 0xbf800000u;
  asm("" : "+s"(f), "+s"(s));
  const bf16x2 first = __builtin_bit_cast(bf16x2, f), second = __builtin_bit_cast(bf16x2, s);
  f32x4 r;
  for (int i = 0; i < 4; i += 2) {
    const bf16x2 h = {hi[i], hi[i + 1]};
    r[i] = __builtin_amdgcn_fdot2_f32_bf16(h, first, x[i], false);
    r[i + 1] = __builtin_amdgcn_fdot2_f32_bf16(h, second, x[i + 1], false);
  }
  return r;
}

template <int NP>
__device__ __forceinline__ Parts<NP> parts_of(const f32x4& a, const f32x4& b) {
  Parts<NP> r;
  const bf16x4 ah = rounded(a), bh = rounded(b);
  r.p[0] = join(ah, bh);
  if constexpr (NP >= 2) {
    const f32x4 ar = rest_of(a, ah), br = rest_of(b, bh);
    const bf16x4 am = rounded(ar), bm = rounded(br);
    r.p[1] = join(am, bm);
    if constexpr (NP == 3) r.p[2] = join(rounded(rest_of(ar, am)), rounded(rest_of(br, bm)));
  }
  return r;
}

// Product of operands in NA and NB parts, every part 2^-8 of the one before, with the
// terms above 2^-24.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Parts<NA>& a, const Parts<NB>& b, f32x4 c) {
  for (int i = NA - 1; i >= 0; --i)
    for (int j = NB - 1; j >= 0; --j)
      if (i + j < kParts) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[j], c, 0, 0, 0);
  return c;
}

template <int D, typename T>
struct Dims16 {
  static constexpr int NP = sizeof(T) == 2 && __is_same(T, bf16) ? 1 : 2;   // parts of q and k
  static constexpr int DP = D < 32 ? 32 : D;
  static constexpr int RB = 2 * DP;              // bytes of a row in LDS
  static constexpr int CPR = RB / 16;            // 16-byte units of a row
  static constexpr int KB = DP / 32;
  static constexpr int RT = DP / 16;              // tiles of 16 key channels of a state
  static constexpr int MAT = C * RB;             // bytes of one part of q, k or v
};

// A row's 16-byte units are permuted within it (exclusive or with a number that
// depends on the row), so that the 16 rows an operand takes from a column of
// units fall on different banks.
template <int RB>
__device__ __forceinline__ int unit_at(int row, int unit) {
  return row * RB + ((unit ^ ((row / (256 / RB)) & (RB / 16 - 1))) << 4);
}

// An operand (i, tb) of a lower triangle, i = 0 .. 3, tb <= i / 2, is 16 x 32: 16
// bytes a lane, 1024 in all (kTri for a triangle), in the order lanes hold it.

// Depth over key channels runs, within every 32, in their own order: a lane's eight
// values of an operand are 16 consecutive bytes of a row.  So the 16 rows of state
// tile t that a lane's accumulators hold, 4 g + e, are key channels
// 32 (t / 2) + 8 g + 4 (t % 2) + e, and two tiles are an operand as they stand.
//
// Where a lane reads: `row` for row_operand and `col` for column_operand, of tile 0.
// Other tiles differ by whole 16 rows and in the bits of the unit, which commute
// with the permutation.
struct At {
  int row, col;
};
template <int RB>
__device__ __forceinline__ At lane_at(int lane) {
  const int g = lane >> 4, c = lane & 15;
  return {unit_at<RB>(c, g), unit_at<RB>(4 * g + (c >> 2), c & 3)};
}
// Operand whose row lane % 16 is row 16 i + lane % 16 of x, depth 32 kb ..
template <int RB>
__device__ __forceinline__ bf16x8 row_operand(const uint8_t* x, int i, int kb, At at) {
  return *reinterpret_cast<const bf16x8*>(x + 16 * i * RB + (at.row ^ kb << 6));
}
__device__ __forceinline__ s16x4 read_transposed(const uint8_t* x) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(const_cast<uint8_t*>(x)));
}
// Operand whose rows are the key channels of state tile t, depth tokens 32 tb ..
template <int RB>
__device__ __forceinline__ bf16x8 column_operand(const uint8_t* x, int tb, int t, At at) {
  x += 32 * tb * RB + (at.col ^ (t >> 1) << 6) + (t & 1) * 8;
  return join(__builtin_bit_cast(bf16x4, read_transposed(x)), __builtin_bit_cast(bf16x4, read_transposed(x + 16 * RB)));
}
// Tokens 16 i + 4 g .. + 3 (g = lane / 16) of value column 16 t + lane % 16 of x.
template <int RB>
__device__ __forceinline__ s16x4 value_piece(const uint8_t* x, int i, int t, int lane) {
  const int g = lane >> 4, c = lane & 15;
  return read_transposed(x + 16 * i * RB + (unit_at<RB>(4 * g + (c >> 2), (c & 3) >> 1) ^ (2 * t) << 4) + (c & 1) * 8);
}
__device__ __forceinline__ bf16x8 stored_operand(const uint8_t* x, int n, int lane) {
  return *reinterpret_cast<const bf16x8*>(x + n * 1024 + lane * 16);
}
// Index of operand (i, tb) of a lower triangle.
__device__ constexpr int tri(int i, int tb) { return i < 2 ? i : 2 * (i - 1) + tb; }

// Half `half` of operand n of a triangle, its parts kTri bytes apart.
__device__ __forceinline__ void store_parts(uint8_t* x, int n, int half, f32x4 y, int lane) {
  const int at = n * 1024 + lane * 16 + half * 8;
  for (int p = 0; p < kParts; ++p) {
    const bf16x4 h = rounded(y);
    *reinterpret_cast<bf16x4*>(x + p * kTri + at) = h;
    if (p + 1 < kParts) y = rest_of(y, h);
  }
}
// Operand n of a triangle.
__device__ __forceinline__ Parts<kParts> stored_parts(const uint8_t* x, int n, int lane) {
  Parts<kParts> r;
  for (int p = 0; p < kParts; ++p) r.p[p] = stored_operand(x + p * kTri, n, lane);
  return r;
}

__device__ __forceinline__ f32x4 floats_of(const s16x4& x, bf16) {
  return widened(__builtin_bit_cast(bf16x4, x));
}
__device__ __forceinline__ f32x4 floats_of(const s16x4& x, f16) {
  typedef f16 f16x4 __attribute__((ext_vector_type(4)));
  return __builtin_convertvector(__builtin_bit_cast(f16x4, x), f32x4);
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Units u0 .. u0 + N - 1 of the rows of a chunk of x (q, k or v of a head), on the
// way from memory to LDS in the registers of THREADS threads: all loads are under
// way before the first is waited for.  A thread has a unit of every THREADS / N'th
// row, 32-bit offsets apart (strides are at most 2^24 elements).
// Past `count` tokens and past D channels the last valid ones are read, and zeros
// are stored.
template <int D, typename T, int N, int THREADS, int RB = Dims16<D, T>::RB>
struct Rows {
  using S = Dims16<D, T>;
  static constexpr int CPR = RB / 16;
  static constexpr int L = C * N / THREADS;
  static constexpr int STEP = THREADS / N;       // a power of two, as N is
  u32x4 raw[L];
  __device__ __forceinline__ void load(const T* x, int64_t stride, int count, int u0, int tid) {
    const uint8_t* base = reinterpret_cast<const uint8_t*>(x);
    const int unit = min(u0 + tid % N, D / 8 - 1);
    const uint32_t s = static_cast<uint32_t>(stride) * 2;
    for (int j = 0; j < L; ++j)
      raw[j] = *reinterpret_cast<const u32x4*>(base + (min(tid / N + j * STEP, count - 1) * s + unit * 16));
  }
  // Into rows of RB bytes.  SPLIT: in two bfloat16 parts, the second S::MAT bytes after
  // the first.
  template <bool SPLIT>
  __device__ __forceinline__ void store(uint8_t* lds, int count, int tid) {
    if (count < C || N * 8 > D)
      for (int j = 0; j < L; ++j)
        if (tid / N + j * STEP >= count || tid % N * 8 >= D) raw[j] = u32x4{};
    const int to0 = unit_at<RB>(tid / N, tid % N);
    for (int j = 0; j < L; ++j) {
      // tid / N < STEP, so the row's number in the permutation is that of its two parts, joined
      uint8_t* to = lds + j * STEP * RB + (to0 ^ ((j * STEP / (256 / RB)) & (CPR - 1)) << 4);
      if constexpr (SPLIT) {
        typedef f16 f16x8 __attribute__((ext_vector_type(8)));
        typedef float f32x8 __attribute__((ext_vector_type(8)));
        const f32x8 y = __builtin_convertvector(__builtin_bit_cast(f16x8, raw[j]), f32x8);
        const bf16x8 hi = __builtin_convertvector(y, bf16x8);
        *reinterpret_cast<bf16x8*>(to) = hi;
        *reinterpret_cast<bf16x8*>(to + S::MAT) = __builtin_convertvector(y - __builtin_convertvector(hi, f32x8), bf16x8);
      } else {
        *reinterpret_cast<u32x4*>(to) = raw[j];
      }
    }
  }
};

// One word of every 128 bytes of a chunk's rows of x, read while an earlier chunk is
// computed so that the rows come from L2 when they are staged: two or three
// registers, where the rows themselves would take 48.
template <int D, typename T, int THREADS>
struct Touch {
  static constexpr int LINES = (2 * D + 127) / 128, L = (C * LINES + THREADS - 1) / THREADS;
  uint32_t word[L] = {};
  __device__ __forceinline__ void start(const T* x, int64_t stride, int count, int tid) {
    for (int j = 0; j < L; ++j) {
      const int i = tid + j * THREADS;
      if (i < C * LINES) word[j] = *reinterpret_cast<const uint32_t*>(x + min(i / LINES, count - 1) * stride + i % LINES * 64);
    }
  }
  __device__ __forceinline__ void end() {
    for (int j = 0; j < L; ++j) asm volatile("" ::"v"(word[j]));
  }
};

// What a chunk's retentions and betas come to, in LDS.
struct Rates {
  double lg[C];      // log2 G
  float grow[C];     // G_t
  float left[C];     // G_C / G_t
  float beta[C];
};

// One wave: the chunk's log2 G as a running sum in binary64, so that ratios of
// retentions far into a fast-forgetting chunk keep binary32 accuracy.  Its terms are
// binary32 logarithms, good to a unit in their last place also next to 1 (the
// binary32 kernel, which has the time, takes them in binary64).  A retention of 0
// or below 2^-126 counts as 2^-200, which leaves nothing in binary32.  Past `count`
// tokens: retention 1, beta 0.
__device__ __forceinline__ void set_rates(Rates& r, float gate, float beta, int count, int lane) {
  double x = 0.0;
  if (lane < count) {
    const float y = __builtin_amdgcn_logf(gate);
    x = y < -200.0f ? -200.0 : static_cast<double>(y);
  }
  for (int s = 1; s < 64; s <<= 1) {
    const double y = __shfl_up(x, s);
    if (lane >= s) x += y;
  }
  const double all = __shfl(x, 63);
  r.lg[lane] = x;
  r.grow[lane] = __builtin_amdgcn_exp2f(static_cast<float>(x));
  r.left[lane] = __builtin_amdgcn_exp2f(static_cast<float>(all - x));
  r.beta[lane] = lane < count ? beta : 0.0f;
}

// Diagonal blocks of B, later their inverses, in rows of 20.
struct Scratch {
  float diag[4][16 * 20];
};

// Block (i, j) of A and of the system for U into LDS, one wave, both as operands in
// parts (`lt`, `la`).  With
// B = diag(b) B', U comes from block rows of 16 tokens in turn,
//   U_i = D_i (R_i - sum_{j < i} B'_ij U_j),  D_i = (I + B_ii)^-1 diag(b_i),
// so the system is stored as -B'_ij below the diagonal and D_i on it.  The inverse
// is found by forward substitution, a column for every lane of 16 (four times over).
template <int D, typename T, bool DELTA, bool DIAGONAL>
__device__ __forceinline__ void chunk_tile(const uint8_t* lk, const uint8_t* lq, const Rates& r, Scratch* sc,
                                           uint8_t* la, uint8_t* lt, int i, int j, int lane) {
  using S = Dims16<D, T>;
  const At at = lane_at<S::RB>(lane);
  const int g = lane >> 4, c = lane & 15;
  // rows: key token 16 j + 4 g + e, column: token 16 i + c
  f32x4 kk = {}, qk = {};
  for (int kb = 0; kb < S::KB; ++kb) {
    Parts<S::NP> ki, qi, kj;
    for (int x = 0; x < S::NP; ++x) {
      kj.p[x] = row_operand<S::RB>(lk + x * S::MAT, j, kb, at);
      qi.p[x] = row_operand<S::RB>(lq + x * S::MAT, i, kb, at);
      if constexpr (DELTA) ki.p[x] = DIAGONAL ? kj.p[x] : row_operand<S::RB>(lk + x * S::MAT, i, kb, at);
    }
    qk = mma(kj, qi, qk);
    if constexpr (DELTA) kk = mma(kj, ki, kk);
  }
  settle();
  const double li = r.lg[16 * i + c];
  f32x4 ratio;
  for (int e = 0; e < 4; ++e) {
    const float x = __builtin_amdgcn_exp2f(static_cast<float>(li - r.lg[16 * j + 4 * g + e]));
    ratio[e] = !DIAGONAL || 4 * g + e <= c ? x : 0.0f;
  }
  const int to = tri(i, j >> 1);
  store_parts(la, to, j & 1, qk * ratio, lane);
  if constexpr (DELTA && !DIAGONAL) {
    store_parts(lt, to, j & 1, -kk * ratio, lane);
  } else if constexpr (DELTA) {
    // the wave's own LDS accesses are in order; of B only what is below the diagonal is read
    float* d = sc->diag[i];
    *reinterpret_cast<f32x4*>(d + c * 20 + 4 * g) = kk * ratio * r.beta[16 * i + c];
    wave_order();
    float x[16];
    for (int q = 0; q < 8; ++q) {      // two rows at a time: registers
      f32x4 row[2][4];
      for (int ii = 0; ii < 2; ++ii)
        for (int b = 0; b <= q / 2; ++b) row[ii][b] = *reinterpret_cast<const f32x4*>(d + (2 * q + ii) * 20 + 4 * b);
      for (int ii = 0; ii < 2; ++ii) {
        float s = 2 * q + ii == c ? 1.0f : 0.0f;
        for (int jj = 0; jj < 2 * q + ii; ++jj) s = fmaf(-row[ii][jj >> 2][jj & 3], x[jj], s);
        x[2 * q + ii] = s;
      }
      in_order();
    }
    wave_order();
    if (g == 0)
      for (int ii = 0; ii < 16; ++ii) d[ii * 20 + c] = x[ii];
    wave_order();
    const f32x4 inv = *reinterpret_cast<const f32x4*>(d + c * 20 + 4 * g) *
                      *reinterpret_cast<const f32x4*>(&r.beta[16 * i + 4 * g]);
    store_parts(lt, to, j & 1, inv, lane);
  }
  if (DIAGONAL && (i & 1) == 0) {      // beside the diagonal
    store_parts(la, to, 1, f32x4{}, lane);
    if constexpr (DELTA) store_parts(lt, to, 1, f32x4{}, lane);
  }
  in_order();
}

// The ten blocks (i, j), j <= i < 4, of a chunk's lower triangles, dealt out to the
// waves of a workgroup.
template <int D, typename T, bool DELTA, int NW>
__device__ __forceinline__ void chunk_tiles(const uint8_t* lk, const uint8_t* lq, const Rates& r, Scratch* sc,
                                            uint8_t* la, uint8_t* lt, int wave, int lane) {
  static_assert(NW == 4 || NW == 8, "four or eight waves");
  if (wave < 4) chunk_tile<D, T, DELTA, true>(lk, lq, r, sc, la, lt, wave, wave, lane);
  const int w = NW == 8 ? wave - 4 : wave;
  if (w >= 0) {
    const int i = w == 0 ? 3 : w == 1 ? 1 : w == 2 ? 2 : 3, j = w == 0 ? 0 : w == 1 ? 0 : w == 2 ? 1 : 2;
    chunk_tile<D, T, DELTA, false>(lk, lq, r, sc, la, lt, i, j, lane);
    if (w < 2) chunk_tile<D, T, DELTA, false>(lk, lq, r, sc, la, lt, w == 0 ? 2 : 3, w, lane);
  }
}

// LDS.  FUSED: `rates` for this chunk and the next one; HEAD: G, G_C / G, A and the
// system lie as they do in the workspace.  V takes the place of Q, at the price of a
// barrier, where two workgroups fit a compute unit only so (FUSED, delta rule: bfloat16
// at D = 128, binary16 at D = 64).
template <int D, typename T, bool DELTA, int COLS, bool FUSED, bool HEAD = !FUSED>
struct Lds16 {
  using S = Dims16<D, T>;
  static constexpr int RBV = 2 * COLS < 64 ? 64 : 2 * COLS;      // bytes of a row of v
  static constexpr int K = 0;
  static constexpr int Q = K + S::NP * S::MAT;
  static constexpr int REST = (HEAD ? 2 * C * 4 : 0) + (DELTA ? 2 : 1) * kParts * kTri +
                              (FUSED ? 2 * static_cast<int>(sizeof(Rates)) + (DELTA ? static_cast<int>(sizeof(Scratch)) : 0) : 0);
  static constexpr bool V_OVER_Q = FUSED && !HEAD && C * RBV <= S::NP * S::MAT &&
                                   Q + S::NP * S::MAT + C * RBV + REST > kLds / 2 && Q + S::NP * S::MAT + REST <= kLds / 2;
  static constexpr int V = V_OVER_Q ? Q : Q + S::NP * S::MAT;
  static constexpr int BLOCK = Q + S::NP * S::MAT + (V_OVER_Q ? 0 : C * RBV);
  static constexpr int A = BLOCK + (HEAD ? 2 * C * 4 : 0);
  static constexpr int TT = A + kParts * kTri;
  static constexpr int RATES = TT + (DELTA ? kParts * kTri : 0);
  static constexpr int SCRATCH = RATES + 2 * static_cast<int>(sizeof(Rates));
  static constexpr int BYTES = BLOCK + REST;
};

// Workgroups are dealt out to the chip's 8 dies in turn, each with an L2 of its own.
// Those that read the same q and k (`n` of them: value heads of a key head, column
// parts of a head) are numbered 8 apart, so that they meet in one.
__device__ __forceinline__ uint32_t die_order(uint32_t block, uint32_t total, uint32_t n) {
  const uint32_t set = 8 * n, whole = total / set * set, w = block % set;
  return block < whole ? block - w + (w % 8) * n + w / 8 : block;
}

// The chunk matrices of every (chunk, head), for k_linear16_walk<.., false>.  Bound by
// latency; two workgroups a compute unit (one for binary16, whose parts take the LDS).
template <int D, typename T, bool DELTA>
__global__ void __launch_bounds__(kThreads) k_linear16_chunks(LinearArgs p) {
  using S = Dims16<D, T>;
  using L = Lds16<D, T, DELTA, 16, true, true>;      // no v
  extern __shared__ __align__(16) uint8_t lds16[];
  Rates& rates = *reinterpret_cast<Rates*>(lds16 + L::RATES);
  Scratch* sc = reinterpret_cast<Scratch*>(lds16 + L::SCRATCH);
  const uint32_t block = die_order(blockIdx.x, gridDim.x, p.rep);
  const int h = block % p.H;
  const int64_t w = block / p.H;
  const int b = owner(p, w, C);
  const Span r = request_span(p, b);
  const int64_t c = w - (r.first / C + b);
  if (c < 0 || c * C >= r.count) return;
  const int64_t first = r.first + c * C;
  const int count = min(C, static_cast<int>(r.count - c * C));
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const T* k = static_cast<const T*>(p.k) + first * p.k_stride + (h / p.rep) * D;
  const T* q = static_cast<const T*>(p.q) + first * p.q_stride + (h / p.rep) * D;
  Rows<D, T, S::CPR, kThreads> kr, qr;
  kr.load(k, p.k_stride, count, 0, tid);
  qr.load(q, p.q_stride, count, 0, tid);
  if (wave == 0) {
    const int64_t at = (first + min(lane, count - 1)) * p.H + h;
    set_rates(rates, p.gate[at], DELTA ? p.beta[at] : 0.0f, count, lane);
  }
  kr.template store<S::NP == 2>(lds16 + L::K, count, tid);
  qr.template store<S::NP == 2>(lds16 + L::Q, count, tid);
  __syncthreads();
  chunk_tiles<D, T, DELTA, 4>(lds16 + L::K, lds16 + L::Q, rates, sc, lds16 + L::A, lds16 + L::TT, wave, lane);
  __syncthreads();
  if (tid < 2 * C) reinterpret_cast<float*>(lds16 + L::BLOCK)[tid] = (tid < C ? rates.grow : rates.left)[tid % C];
  __syncthreads();
  uint8_t* ws = p.workspace + (w * p.H + h) * block_bytes(DELTA);
  for (int i = tid * 16; i < block_bytes(DELTA); i += kThreads * 16)
    *reinterpret_cast<u32x4*>(ws + i) = *reinterpret_cast<const u32x4*>(lds16 + L::BLOCK + i);
}

// The request that comes `nth` by length, longest first, among up to 64 (beyond
// that, where a chip full of workgroups evens lengths out by itself, in their own
// order): 32768 tokens of 16 requests of 500 to 3500 take 1.14 ms in their own order,
// with long ones starting last, and 0.83 ms so; 8192 of 8, 378 and 306 us.
__device__ __forceinline__ int nth_longest(const LinearArgs& p, int nth, int lane) {
  if (p.batch == 1 || p.batch > 64) return nth;
  const int n = lane < p.batch ? request_span(p, lane).count : -1;
  int rank = 0;
  for (int j = 0; j < p.batch; ++j) {
    const int m = __builtin_amdgcn_readlane(n, j);
    rank += m > n || (m == n && j < lane) ? 1 : 0;
  }
  return __builtin_ctzll(__ballot(lane < p.batch && rank == nth));
}

// Walks a request's chunks in order for 16 NCT NW value columns of one head.
// FUSED: all columns of the head in one workgroup, which computes the chunk
// matrices itself; otherwise they come from k_linear16_chunks.
//
// A long prompt of few heads under the additive rule is walked in segments of
// p.segment chunks at once: what a segment adds to the state does not depend on the
// state it starts from, which only fades.  PASS 1 leaves every segment's own state
// and retention in the workspace, k_linear_join turns them into the states that
// segments start from, and PASS 2 computes the outputs.  One 16384-token prompt of
// 32 heads: 1199 us in 256 chunks one after another, 288 us in segments.
//
// At D = 128 the delta rule takes 456 matrix instructions of 16 cycles a chunk from
// each of four waves with 32 columns (fewer, wider waves read q and k from LDS half as
// often as eight with 16, and those spilled: 381 us against 225 for 512 pairs of 1024
// tokens, both with operands in two parts, where this takes 273 now); the additive rule
// fits 128 registers with eight waves (157 against 162 us, in two parts as well).
// Bound by latency: with two workgroups a compute unit the matrix units are busy 44 %
// and the vector units 46 % of the time, memory 27 % of its rate; the chain of a chunk
// (staging, blocks and their inverses, K M and Q M, U, O, the state) has three barriers,
// four where V takes Q's place, and leaves two waves a SIMD too little to overlap.  32768
// tokens of 16 requests and 48 heads take 780 to 830 us, 3.5 to 3.8 times what copying
// their bytes takes.
template <int D, typename T, bool DELTA, int NCT, int NW, bool FUSED, int PASS>
__global__ void __launch_bounds__(64 * NW, FUSED && __is_same(T, bf16) ? NW / 2 : 1) k_linear16_walk(LinearArgs p) {
  using S = Dims16<D, T>;
  constexpr int NP = S::NP;
  constexpr int UP = DELTA ? kParts : NP;      // the additive rule's U is V as it came
  constexpr int COLS = 16 * NCT * NW;
  constexpr int THREADS = 64 * NW;
  using L = Lds16<D, T, DELTA, COLS, FUSED>;
  constexpr int SPLIT = D / COLS;
  extern __shared__ __align__(16) uint8_t lds16[];
  uint8_t* lk = lds16 + L::K;
  uint8_t* lq = lds16 + L::Q;
  uint8_t* lv = lds16 + L::V;
  uint8_t* la = lds16 + L::A;
  uint8_t* lt = lds16 + L::TT;
  Rates* all_rates = reinterpret_cast<Rates*>(lds16 + L::RATES);
  Scratch* sc = reinterpret_cast<Scratch*>(lds16 + L::SCRATCH);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t block = die_order(blockIdx.x, gridDim.x, p.rep * SPLIT);
  const int part = block % SPLIT;
  const int h = (block / SPLIT) % p.H;
  int b = 0;
  int64_t segment = block / (SPLIT * p.H);
  if constexpr (PASS == 0) {
    b = nth_longest(p, static_cast<int>(segment), lane);
  } else {
    b = owner(p, segment, p.segment * C);
  }
  const int ct0 = part * (COLS / 16) + wave * NCT;      // first column tile of the wave
  Span r = request_span(p, b);
  if constexpr (PASS != 0) {
    const int64_t skip = (segment - (r.first / (p.segment * C) + b)) * p.segment * C;
    if (skip < 0 || skip >= r.count) return;
    r = {r.first + skip, static_cast<int32_t>(min(r.count - skip, static_cast<int64_t>(p.segment) * C))};
  }
  const int slot = p.slot_ids[b];
  T* o = static_cast<T*>(p.o) + r.first * p.o_stride + h * D;
  if (slot < 0 || slot >= p.num_slots) {
    if constexpr (PASS == 1) return;
    for (int t = tid / COLS; t < r.count; t += THREADS / COLS > 0 ? THREADS / COLS : 1)
      for (int j = tid % COLS; j < COLS; j += THREADS) o[t * p.o_stride + part * COLS + j] = static_cast<T>(__builtin_nanf(""));
    return;
  }
  const T* v = static_cast<const T*>(p.v) + r.first * p.v_stride + h * D;
  const T* k = static_cast<const T*>(p.k) + r.first * p.k_stride + (h / p.rep) * D;
  const T* q = static_cast<const T*>(p.q) + r.first * p.q_stride + (h / p.rep) * D;
  float* state = (PASS == 0 ? p.state + (static_cast<int64_t>(slot) * p.H + h) * D * D
                            : reinterpret_cast<float*>(p.workspace) + (segment * p.H + h) * (D * D + kSegmentHead)) + 16 * ct0;

  // column 16 (ct0 + n) + lane % 16; tile i holds key channels 32 (i / 2) + 8 g + 4 (i % 2) + e
  f32x4 m[NCT][S::RT] = {};
  if (PASS == 2 || (PASS == 0 && p.resume != nullptr && p.resume[b] != 0)) {
    const int l = fresh(lane), g = l >> 4, at = g * 8 * D + (l & 15);
    if (8 * g < D)
      for (int n = 0; n < NCT; ++n)
        for (int i = 0; i < S::RT; ++i)
          for (int e = 0; e < 4; ++e) m[n][i][e] = state[at + (32 * (i / 2) + 4 * (i % 2) + e) * D + 16 * n];
  }

  constexpr int VU = COLS / 8;      // units of the workgroup's columns
  float gate = 0.0f, beta = 0.0f;
  // FUSED: the next chunk's rows are touched while this one is computed.  Otherwise a
  // wave has registers enough to hold all of the next chunk's data.
  Touch<D, T, THREADS> kt, qt, vt;
  Rows<D, T, S::CPR, THREADS> kr, qr;
  Rows<D, T, VU, THREADS, L::RBV> vr;
  constexpr int BU = block_bytes(DELTA) / 16, BL = (BU + THREADS - 1) / THREADS;
  u32x4 br[BL];
  const uint8_t* ws = p.workspace + ((r.first / C + b) * p.H + h) * block_bytes(DELTA);
  auto load_rows = [&](int64_t t0) __attribute__((always_inline)) {
    const int t = fresh(tid), n = static_cast<int>(min(static_cast<int64_t>(C), r.count - t0));
    kr.load(k + t0 * p.k_stride, p.k_stride, n, 0, t);
    if constexpr (PASS != 1) qr.load(q + t0 * p.q_stride, p.q_stride, n, 0, t);
    vr.load(v + t0 * p.v_stride, p.v_stride, n, part * VU, t);
    if constexpr (!FUSED)
      for (int j = 0; j < BL; ++j)
        br[j] = *reinterpret_cast<const u32x4*>(ws + t0 / C * p.H * block_bytes(DELTA) + min(t + j * THREADS, BU - 1) * 16);
  };
  if (!FUSED && r.count > 0) load_rows(0);
  constexpr int RATES_WAVE = NW - 2;      // a wave with few blocks sets the next chunk's rates
  if (FUSED && r.count > 0 && wave == RATES_WAVE) {
    const int64_t token = (r.first + min(lane, r.count - 1)) * p.H + h;
    gate = p.gate[token];
    if constexpr (DELTA) beta = p.beta[token];
    set_rates(all_rates[0], gate, beta, min(C, r.count), lane);
  }
  float faded = 1.0f;     // the product of the retentions so far
  for (int c = 0; c * C < r.count; ++c) {
    const int count = min(C, r.count - c * C);
    const int64_t t0 = static_cast<int64_t>(c) * C;
    const bool more = t0 + C < r.count;
    Rates& rates = all_rates[c & 1];
    const float* grow = FUSED ? rates.grow : reinterpret_cast<const float*>(lds16 + L::BLOCK);
    const float* left = FUSED ? rates.left : grow + C;
    if constexpr (FUSED) {
      kt.end();
      qt.end();
      vt.end();
      load_rows(t0);
    }
    __syncthreads();
    {
      const int t = fresh(tid);
      kr.template store<NP == 2>(lk, count, t);
      if constexpr (PASS != 1) qr.template store<NP == 2>(lq, count, t);
      if constexpr (!FUSED) {
        vr.template store<false>(lv, count, t);
        for (int j = 0; j < BL; ++j)
          if (t + j * THREADS < BU) *reinterpret_cast<u32x4*>(lds16 + L::BLOCK + (t + j * THREADS) * 16) = br[j];
      }
    }
    if constexpr (FUSED) {
      const bool next = more && wave == RATES_WAVE;
      if (next) {
        const int64_t token = (r.first + t0 + C + min(lane, r.count - (c + 1) * C - 1)) * p.H + h;
        gate = p.gate[token];
        if constexpr (DELTA) beta = p.beta[token];
      }
      __syncthreads();
      if constexpr (PASS != 1) chunk_tiles<D, T, DELTA, NW>(lk, lq, rates, sc, la, lt, wave, fresh(lane));
      if (next) set_rates(all_rates[(c + 1) & 1], gate, beta, min(C, r.count - (c + 1) * C), lane);
      if (more) {
        const int t = fresh(tid), n = min(C, r.count - (c + 1) * C);
        kt.start(k + (t0 + C) * p.k_stride, p.k_stride, n, t);
        if constexpr (PASS != 1) qt.start(q + (t0 + C) * p.q_stride, p.q_stride, n, t);
        vt.start(v + (t0 + C) * p.v_stride, p.v_stride, n, t);
      }
    } else {
      __syncthreads();
      if (more) load_rows(t0 + C);
    }

    // K M and (transposed: rows value columns, columns tokens, so that a lane stores
    // 4 neighbours) Q M, the state split into its parts once for both
    f32x4 u[NCT][4] = {}, y[NCT][4] = {};
    if constexpr (PASS != 1) {
    const At at = lane_at<S::RB>(fresh(lane));
    for (int kb = 0; kb < S::KB; ++kb) {
      Parts<kParts> mf[NCT];
      for (int n = 0; n < NCT; ++n) mf[n] = parts_of<kParts>(m[n][2 * kb], m[n][2 * kb + 1]);
      for (int i = 0; i < 4; ++i) {
        Parts<NP> a;
        if constexpr (DELTA) {
          for (int x = 0; x < NP; ++x) a.p[x] = row_operand<S::RB>(lk + x * S::MAT, i, kb, at);
          for (int n = 0; n < NCT; ++n) u[n][i] = mma(a, mf[n], u[n][i]);
        }
        for (int x = 0; x < NP; ++x) a.p[x] = row_operand<S::RB>(lq + x * S::MAT, i, kb, at);
        for (int n = 0; n < NCT; ++n) y[n][i] = mma(mf[n], a, y[n][i]);
      }
      in_order();
    }
    }
    settle();
    if constexpr (FUSED) {
      if constexpr (L::V_OVER_Q) __syncthreads();      // Q has been read
      vr.template store<false>(lv, count, fresh(tid));
      __syncthreads();      // V, A and the system for U
    }
    Parts<UP> uf[NCT][2];
    {
      const int l = fresh(lane), g = l >> 4;
      for (int n = 0; n < NCT; ++n)
        for (int i = 0; i < 4; ++i) {
          const f32x4 x = floats_of(value_piece<L::RBV>(lv, i, wave * NCT + n, l), T{});
          if constexpr (DELTA) u[n][i] = x - *reinterpret_cast<const f32x4*>(&grow[16 * i + 4 * g]) * u[n][i];
          else u[n][i] = x;
        }
      const f32x4 none = {};
      if constexpr (DELTA) {
        Parts<kParts> s = stored_parts(lt, tri(0, 0), l);
        for (int n = 0; n < NCT; ++n) u[n][0] = mma(s, parts_of<kParts>(u[n][0], none), none);
        s = stored_parts(lt, tri(1, 0), l);
        for (int n = 0; n < NCT; ++n) u[n][1] = mma(s, parts_of<kParts>(u[n][0], none), u[n][1]);
        for (int n = 0; n < NCT; ++n) u[n][1] = mma(s, parts_of<kParts>(none, u[n][1]), none);
        for (int n = 0; n < NCT; ++n) uf[n][0] = parts_of<kParts>(u[n][0], u[n][1]);
        s = stored_parts(lt, tri(2, 0), l);
        for (int n = 0; n < NCT; ++n) u[n][2] = mma(s, uf[n][0], u[n][2]);
        s = stored_parts(lt, tri(3, 0), l);
        for (int n = 0; n < NCT; ++n) u[n][3] = mma(s, uf[n][0], u[n][3]);
        s = stored_parts(lt, tri(2, 1), l);
        for (int n = 0; n < NCT; ++n) u[n][2] = mma(s, parts_of<kParts>(u[n][2], none), none);
        s = stored_parts(lt, tri(3, 1), l);
        for (int n = 0; n < NCT; ++n) u[n][3] = mma(s, parts_of<kParts>(u[n][2], none), u[n][3]);
        for (int n = 0; n < NCT; ++n) u[n][3] = mma(s, parts_of<kParts>(none, u[n][3]), none);
        for (int n = 0; n < NCT; ++n) uf[n][1] = parts_of<kParts>(u[n][2], u[n][3]);
      } else {
        for (int n = 0; n < NCT; ++n)
          for (int tb = 0; tb < 2; ++tb) uf[n][tb] = parts_of<UP>(u[n][2 * tb], u[n][2 * tb + 1]);
      }
      in_order();
    }
    if constexpr (PASS != 1) {
      const int l = fresh(lane), g = l >> 4, cl = l & 15;
      for (int i = 0; i < 4; ++i) {
        const float f = grow[16 * i + cl];
        for (int n = 0; n < NCT; ++n) y[n][i] *= f;
        for (int tb = 0; tb <= i / 2; ++tb) {
          const Parts<kParts> a = stored_parts(la, tri(i, tb), l);
          for (int n = 0; n < NCT; ++n) y[n][i] = mma(uf[n][tb], a, y[n][i]);
        }
      }
      settle();
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * i + cl;
        if (t < count)
          for (int n = 0; n < NCT; ++n) {
            typedef T t16x4 __attribute__((ext_vector_type(4)));
            *reinterpret_cast<t16x4*>(o + (t0 + t) * p.o_stride + 16 * (ct0 + n) + 4 * g) =
                __builtin_convertvector(y[n][i], t16x4);
          }
      }
    }
    in_order();
    const int l = fresh(lane), g = l >> 4;
    const At at = lane_at<S::RB>(l);
    Parts<kParts> wf[NCT][2];
    const float all = grow[C - 1];
    faded *= all;
    for (int n = 0; n < NCT; ++n)
      for (int tb = 0; tb < 2; ++tb)
        wf[n][tb] = parts_of<kParts>(u[n][2 * tb] * *reinterpret_cast<const f32x4*>(&left[32 * tb + 4 * g]),
                                u[n][2 * tb + 1] * *reinterpret_cast<const f32x4*>(&left[32 * tb + 16 + 4 * g]));
    for (int i = 0; i < S::RT; ++i) {
      for (int n = 0; n < NCT; ++n) m[n][i] *= all;
      for (int tb = 0; tb < 2; ++tb) {
        Parts<NP> a;
        for (int x = 0; x < NP; ++x) a.p[x] = column_operand<S::RB>(lk + x * S::MAT, tb, i, at);
        for (int n = 0; n < NCT; ++n) m[n][i] = mma(a, wf[n][tb], m[n][i]);
      }
      if (i % 2) in_order();
    }
    settle();
  }
  if constexpr (PASS == 2) return;
  if (PASS == 1 && tid == 0) state[D * D - 16 * ct0] = faded;
  const int l = fresh(lane), g = l >> 4, at = g * 8 * D + (l & 15);
  if (8 * g < D)      // fewer than 32 channels are padded to 32
    for (int n = 0; n < NCT; ++n)
      for (int i = 0; i < S::RT; ++i)
        for (int e = 0; e < 4; ++e) state[at + (32 * (i / 2) + 4 * (i % 2) + e) * D + 16 * n] = m[n][i][e];
}

// Four neighbouring state values of one (request, head): the states its segments start
// from, in place of their own, and the final state.
template <int D>
__global__ void __launch_bounds__(kThreads) k_linear_join(LinearArgs p) {
  constexpr int PARTS = D * D / (4 * kThreads);
  const int part = blockIdx.x % PARTS, h = blockIdx.x / PARTS % p.H, b = blockIdx.x / PARTS / p.H;
  const Span r = request_span(p, b);
  const int slot = p.slot_ids[b];
  if (slot < 0 || slot >= p.num_slots) return;
  const int at = (part * kThreads + threadIdx.x) * 4;
  float* state = p.state + (static_cast<int64_t>(slot) * p.H + h) * D * D + at;
  f32x4 m = {};
  if (p.resume != nullptr && p.resume[b] != 0) m = *reinterpret_cast<const f32x4*>(state);
  const int64_t base = r.first / (p.segment * C) + b, step = static_cast<int64_t>(p.H) * (D * D + kSegmentHead);
  float* own = reinterpret_cast<float*>(p.workspace) + (base * p.H + h) * (D * D + kSegmentHead);
  for (int64_t s = 0; s * p.segment * C < r.count; ++s, own += step) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(own + at);
    *reinterpret_cast<f32x4*>(own + at) = m;
    m = m * own[D * D] + x;
  }
  *reinterpret_cast<f32x4*>(state) = m;
}

constexpr int step_threads(int d) { return d * d / 4 < kThreads ? d * d / 4 : kThreads; }

// One token: a workgroup owns one (request, head) state; a lane holds 4 columns of
// D / RG rows in registers.  With the decayed state M~,
// u = M~^T k and w = M~^T q (one reduction for both) the new state's readout is
// o = w + (q . k) x with x = b (v - u), or v for the additive rule, so the state
// is read and written once.  Bound by memory: 512 requests of 48 heads of 128 take
// 635 us, 5150 GB/s, what a copy reaches; one request's 48 states take 5.3 us of which
// 1.2 us are its bytes, the rest the latency of one load, two sums and a store.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads) k_linear_step(LinearArgs p) {
  constexpr int LPR = D / 4;
  constexpr int NT = step_threads(D);
  constexpr int RG = NT / LPR;                 // row groups
  constexpr int RPT = D / RG;                  // rows per lane
  static_assert(RPT * RG == D && NT >= D, "every lane has whole rows");
  constexpr int NW = NT / 64;
  __shared__ float qs[D], ks[D];
  __shared__ __align__(16) f32x4 part[NW][2][LPR < 64 ? LPR : 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int h = blockIdx.x % p.H;
  const int64_t b = blockIdx.x / p.H;
  const int j0 = 4 * (tid % LPR);
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
  for (int i = 0; i < RPT; ++i) m[i] = *reinterpret_cast<const f32x4*>(state + (rg + i * RG) * D);
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
  for (int i = 0; i < RPT; ++i) {
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
  for (int i = 0; i < RPT; ++i) *reinterpret_cast<f32x4*>(state + (rg + i * RG) * D) = m[i] + ks[rg + i * RG] * x;
  if (tid < LPR)
    for (int e = 0; e < 4; ++e) o[e] = static_cast<T>(w[e] + qk * x[e]);
}

template <typename K>
hipError_t launch_lds(K* kern, int64_t grid, int threads, int lds, const LinearArgs& a, hipStream_t s) {
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  kern<<<dim3(static_cast<uint32_t>(grid)), threads, lds, s>>>(a);
  return hipGetLastError();
}

template <int D, typename T, bool DELTA, int NW>
hipError_t walk32(const LinearArgs& a, hipStream_t s) {
  const int lds = sizeof(float) * (2 * C * Dims<D>::LD + (DELTA ? 2 : 1) * C * (C + 4));
  return launch_lds(k_linear_walk<D, T, DELTA, NW>, static_cast<int64_t>(a.batch) * a.H * (D / (16 * NW)), 64 * NW, lds, a, s);
}

template <int D, typename T, bool DELTA>
hipError_t prefill_dt(const LinearArgs& a, hipStream_t s) {
  k_linear_chunks<D, T, DELTA><<<dim3(static_cast<uint32_t>(max_chunks(a.total_tokens, a.batch) * a.H)), kThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : walk32<D, T, DELTA, D >= 64 ? 4 : D / 16>(a, s);
}

template <int D, typename T, bool DELTA, int NCT, int NW, bool FUSED, int PASS = 0>
hipError_t walk16(const LinearArgs& a, hipStream_t s) {
  constexpr int COLS = 16 * NCT * NW;
  const int64_t rows = PASS == 0 ? a.batch : max_segments(a.total_tokens, a.batch, a.segment);
  return launch_lds(k_linear16_walk<D, T, DELTA, NCT, NW, FUSED, PASS>, rows * a.H * (D / COLS), 64 * NW,
                    Lds16<D, T, DELTA, COLS, FUSED>::BYTES, a, s);
}

// The walk apart from its chunk matrices, 16 NW columns a workgroup; `waves` is that NW.
template <int D, typename T, bool DELTA, int NW>
hipError_t walk_apart(int waves, const LinearArgs& a, hipStream_t s) {
  static_assert(Lds16<D, T, DELTA, 16 * NW, false>::BYTES == apart_lds(D, Dims16<D, T>::NP, DELTA, NW), "one rule for both");
  constexpr int64_t most = D < 64 ? INT32_MAX : kMostApart;
  if constexpr (apart_waves(D, Dims16<D, T>::NP, DELTA, most) > NW) {
    if (waves > NW) return walk_apart<D, T, DELTA, 2 * NW>(waves, a, s);
  }
  return walk16<D, T, DELTA, 1, NW, false>(a, s);
}

template <int D, typename T, bool DELTA>
hipError_t prefill16(const LinearArgs& a, hipStream_t s) {
  const int64_t tiles = static_cast<int64_t>(a.batch) * a.H;
  if constexpr (D >= 64 && !DELTA) {
    if (a.segment > 0) {
      hipError_t e = walk16<D, T, false, 1, D / 16, true, 1>(a, s);
      if (e != hipSuccess) return e;
      k_linear_join<D><<<dim3(static_cast<uint32_t>(tiles * (D * D / (4 * kThreads)))), kThreads, 0, s>>>(a);
      e = hipGetLastError();
      return e != hipSuccess ? e : walk16<D, T, false, 1, D / 16, true, 2>(a, s);
    }
  }
  if constexpr (ever_apart(D, DELTA)) {
    if (a.apart) {
      const hipError_t e = launch_lds(k_linear16_chunks<D, T, DELTA>, max_chunks(a.total_tokens, a.batch) * a.H, kThreads,
                                      Lds16<D, T, DELTA, 16, true, true>::BYTES, a, s);
      return e != hipSuccess ? e : walk_apart<D, T, DELTA, 1>(apart_waves(D, Dims16<D, T>::NP, DELTA, tiles), a, s);
    }
  }
  if constexpr (D >= 64) return walk16<D, T, DELTA, DELTA ? D / 64 : 1, DELTA ? 4 : D / 16, true>(a, s);
  return hipErrorInvalidValue;
}

template <int D, typename T>
hipError_t step_dt(const LinearArgs& a, hipStream_t s) {
  k_linear_step<D, T><<<dim3(static_cast<uint32_t>(a.batch * a.H)), step_threads(D), 0, s>>>(a);
  return hipGetLastError();
}

template <int D, typename T>
hipError_t prefill_any(const LinearArgs& a, hipStream_t s) {
  if constexpr (sizeof(T) == 4) return a.beta ? prefill_dt<D, T, true>(a, s) : prefill_dt<D, T, false>(a, s);
  else return a.beta ? prefill16<D, T, true>(a, s) : prefill16<D, T, false>(a, s);
}
template <typename T>
hipError_t prefill_t(int d, const LinearArgs& a, hipStream_t s) {
  switch (d) {
    case 16: return prefill_any<16, T>(a, s);
    case 32: return prefill_any<32, T>(a, s);
    case 64: return prefill_any<64, T>(a, s);
    default: return prefill_any<128, T>(a, s);
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
