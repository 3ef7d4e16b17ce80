// Norms around a block, fused with its gate and residual scale, and their
// backward pass.  For one row of n channels:
//   yn = y r1, r1 = 1 / sqrt(mean(y^2) + eps)      (only with a post weight)
//   out = residual + scale silu(gate) post yn      (each factor optional)
//   normed = pre out r2, r2 = 1 / sqrt(mean(out^2) + eps)
// Backward, with D = dout + r2 (d - on mean(d on)), d = pre dnormed, on = out r2:
//   dresidual = D,  dgate = D scale post yn silu'(gate),
//   dy = r1 (e - yn mean(e yn)),  e = D scale silu(gate) post,
//   dpre = sum over rows of dnormed on, dscale of D silu(gate) post yn,
//   dpost of D scale silu(gate) yn.
// The backward pass forms out again from the inputs in fp32: the stored out is
// rounded to its type, and reading residual costs what reading out would.  r1
// and r2 it takes from the forward pass (8 bytes a row).  With u = silu(gate)
// post yn and m = scale u, both of its means then come from sums over the same
// pass: mean(d on) = r2 S1 / n and sum(e yn) = S2 + r2 (S3 - mean(d on) r2 S4),
// S1 = sum d out, S2 = sum m dout, S3 = sum m d, S4 = sum m out: one exchange
// between the threads of a row.
//
// Bound: memory (10 bytes an element forward, 16 backward in bf16), with the
// instruction rate close behind (some 20 and 40 flops an element).  A row lies
// in the registers of one group of threads, so it is read once: narrow rows
// (heads) on 8 to 32 lanes, wide rows on a CTA.  CTAs stay and take row after
// row: a thread's 16-byte pieces of the rows to come travel by cp.async into
// its own places of a shared memory ring, which no other thread reads, so the
// ring needs no barrier; weights and parameter sums stay in registers; fp32
// operations come in pairs.  Rows that do not start on 16 bytes go element by
// element, through shared memory where they are many.
#pragma once

#include "ops.cuh"

namespace dl {

constexpr int kNormMax = 8192;  // channels of a row
// 16-byte units that cover a row of n channels on any address.
template <typename T>
__host__ __device__ constexpr int ahead_units(int n) {
  return (n * static_cast<int>(sizeof(T)) + 15 - static_cast<int>(sizeof(T))) / 16 + 1;
}
constexpr int kNormNarrow = 256;  // threads of a CTA of narrow rows

struct NormArgs {
  const void* y;         // [rows][n] typed
  const void* gate;      // [rows][n] typed or null
  const void* residual;  // [rows][n] typed or null
  const float* post;     // [n] or null
  const float* scale;    // [n] or null
  const float* pre;      // [n] or null
  void* out;             // [rows][n] typed (forward; may be null with pre)
  void* normed;          // [rows][n] typed (forward, with pre)
  const void* dout;      // [rows][n] typed or null (zeros)
  const void* dnormed;   // [rows][n] typed or null (zeros)
  void* dy;              // [rows][n] typed, each null if not wanted
  void* dgate;
  void* dresidual;
  float* stats;          // [rows][2]: r1, r2 (forward: written if not null)
  float* partial;        // [CTAs][3][n]: post, scale, pre sums of the CTA's rows, or null
  const int* slot_idx;   // [rows / groups] or null: rows to skip
  int slots;
  int groups;            // rows here per row of the slot map
  int n;
  int tpr;               // threads of a row
  long long rows;
  float eps;
};

// Whether the slot map (if any: the division is not free) wants this row.
__device__ __forceinline__ bool wanted(const NormArgs& a, long long row) {
  return !a.slot_idx || row_slot(a.slot_idx, a.slots, static_cast<int>(row / a.groups), nullptr, false) >= 0;
}

// Sums K values over the threads of a row.  Narrow: `tpr` (8, 16 or 32) lanes.
// Wide: the whole CTA, through `sm` [2][32][4], whose halves alternate between
// calls so that one barrier a call is enough.
template <int K, bool NARROW>
__device__ __forceinline__ void row_sum(float (&v)[K], int tpr, float (*sm)[32][4], int& turn) {
  if constexpr (!NARROW && K == 4) {
    // four sums in the shuffles of one: halves of the warp keep two values each,
    // quarters one, whose eighth lanes then add up
    const int lane = threadIdx.x % 32, nw = tpr / 32;
    const bool up = lane & 16, odd = lane & 8;
    float a = up ? v[2] : v[0], b = up ? v[3] : v[1];
    a += __shfl_xor_sync(~0u, up ? v[0] : v[2], 16);
    b += __shfl_xor_sync(~0u, up ? v[1] : v[3], 16);
    float c = odd ? b : a;
    c += __shfl_xor_sync(~0u, odd ? a : b, 8);
    c += __shfl_xor_sync(~0u, c, 4);
    c += __shfl_xor_sync(~0u, c, 2);
    c += __shfl_xor_sync(~0u, c, 1);
    float(*s)[4] = sm[turn];
    turn ^= 1;
    if ((lane & 7) == 0) s[threadIdx.x / 32][lane / 8] = c;
    __syncthreads();
    // lane l adds value l % 4 of warps l / 4, l / 4 + 8, ...
    c = 0.f;
    for (int w = lane / 4; w < nw; w += 8) c += s[w][lane % 4];
    c += __shfl_xor_sync(~0u, c, 4);
    c += __shfl_xor_sync(~0u, c, 8);
    c += __shfl_xor_sync(~0u, c, 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __shfl_sync(~0u, c, k);
  } else if constexpr (NARROW) {
    for (int o = tpr / 2; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(~0u, v[k], o);
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(~0u, v[k], o);
    const int lane = threadIdx.x % 32, nw = tpr / 32;
    if (nw == 1) return;
    float(*s)[4] = sm[turn];
    turn ^= 1;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) s[threadIdx.x / 32][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lane < nw ? s[lane][k] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(~0u, v[k], o);
  }
}

// 1 / (1 + 2^(-x log2 e)), the same steps everywhere.
__device__ __forceinline__ float sigmoid(float x) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}

// -- rows that start on 16 bytes ---------------------------------------------------

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// 16 bytes of T as pairs.
template <typename T>
struct Piece {
  static constexpr int V = 16 / sizeof(T), P = V / 2;
  uint4 u;
  __device__ __forceinline__ float2 pair(int i) const {
    const uint32_t* const w = reinterpret_cast<const uint32_t*>(&u);
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void set(int i, float2 x) {
    uint32_t* const w = reinterpret_cast<uint32_t*>(&u);
    if constexpr (sizeof(T) == 4) {
      w[2 * i] = __float_as_uint(x.x);
      w[2 * i + 1] = __float_as_uint(x.y);
    } else {
      const __nv_bfloat162 p = __float22bfloat162_rn(x);
      memcpy(&w[i], &p, 4);
    }
  }
  __device__ __forceinline__ void store(T* p) const { __stcs(reinterpret_cast<uint4*>(p), u); }
};

// One thread's columns of a weight vector, ones where it is absent.
template <int NV, int V>
struct Weights {
  float2 v[NV][V / 2];
  __device__ __forceinline__ void load(const float* p, int lane, int tpr, int n) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * V;
#pragma unroll
      for (int j = 0; j < V / 4; ++j) {
        float4 f = make_float4(1.f, 1.f, 1.f, 1.f);
        if (p && c < n) f = __ldg(reinterpret_cast<const float4*>(p + c) + j);
        v[i][2 * j] = make_float2(f.x, f.y);
        v[i][2 * j + 1] = make_float2(f.z, f.w);
      }
    }
  }
};

// This thread's places for K tensors of S rows: [S][K][NV][threads] of 16 bytes.
template <typename T, int NV, int K, int S>
struct NormRing {
  static constexpr int V = 16 / sizeof(T);
  uint4* place;
  int threads;
  const T* src[K];   // y in place of an absent tensor
  bool present[K];
  __device__ __forceinline__ void set(int k, const void* p, const void* y) {
    present[k] = p != nullptr;
    src[k] = static_cast<const T*>(p ? p : y);
  }
  // Starts bringing a row's pieces, or zeros (outside the row, or absent).
  __device__ __forceinline__ void issue(int s, long long row, bool here, int lane, int tpr, int n) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * V;
      const bool live = here && c < n;
      const long long at = live ? row * n + c : 0;
#pragma unroll
      for (int k = 0; k < K; ++k) copy_async16(place + ((s * K + k) * NV + i) * threads, src[k] + at, live && present[k] ? 16 : 0);
    }
    copy_commit();
  }
  __device__ __forceinline__ Piece<T> get(int s, int k, int i) const {
    return {place[((s * K + k) * NV + i) * threads]};
  }
};

template <typename T, int NV, bool NARROW, bool GATE, bool PRE, int S>
__global__ void __launch_bounds__(NARROW ? kNormNarrow : 512, NARROW ? 4 : 2) norm_ring_kernel(NormArgs a) {
  constexpr int V = 16 / sizeof(T), P = V / 2, K = GATE ? 3 : 2;
  extern __shared__ __align__(16) uint4 ring_places[];
  __shared__ float sm[2][32][4];
  int turn = 0;
  const int lane = NARROW ? static_cast<int>(threadIdx.x) % a.tpr : static_cast<int>(threadIdx.x);
  const int per = NARROW ? kNormNarrow / a.tpr : 1, sub = NARROW ? static_cast<int>(threadIdx.x) / a.tpr : 0;
  const float inv = 1.f / static_cast<float>(a.n);
  const long long step = static_cast<long long>(gridDim.x) * per;
  NormRing<T, NV, K, S> ring{ring_places + threadIdx.x, static_cast<int>(blockDim.x)};
  ring.set(0, a.y, a.y);
  ring.set(1, a.residual, a.y);
  if constexpr (GATE) ring.set(2, a.gate, a.y);
  auto here = [&](long long row) {
    return row < a.rows && wanted(a, row);
  };
  long long first = static_cast<long long>(blockIdx.x) * per;
#pragma unroll
  for (int s = 0; s < S; ++s) ring.issue(s, first + s * step + sub, here(first + s * step + sub), lane, a.tpr, a.n);
  Weights<NV, V> post, scale, pre;
  post.load(a.post, lane, a.tpr, a.n);
  scale.load(a.scale, lane, a.tpr, a.n);
  if constexpr (PRE) pre.load(a.pre, lane, a.tpr, a.n);

  for (int s = 0; first < a.rows; first += step, s = s + 1 == S ? 0 : s + 1) {
    const long long row = first + sub;
    const bool mine = here(row);
    copy_wait<S - 1>();
    Piece<T> y[NV], x[NV], g[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      y[i] = ring.get(s, 0, i);
      x[i] = ring.get(s, 1, i);
      if constexpr (GATE) g[i] = ring.get(s, 2, i);
    }
    ring.issue(s, row + S * step, here(row + S * step), lane, a.tpr, a.n);
    float r1 = 1.f, r2 = 1.f;
    if (a.post) {
      float2 q = both(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < P; ++j) q = fma2(y[i].pair(j), y[i].pair(j), q);
      float ss[1] = {q.x + q.y};
      row_sum<1, NARROW>(ss, a.tpr, sm, turn);
      r1 = rsqrtf(fmaf(ss[0], inv, a.eps));
    }
    float2 o[NV][P], q = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Piece<T> w;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        float2 u = mul2(mul2(y[i].pair(j), both(r1)), post.v[i][j]);
        if constexpr (GATE) {
          const float2 f = g[i].pair(j);
          u = mul2(u, mul2(f, make_float2(sigmoid(f.x), sigmoid(f.y))));
        }
        o[i][j] = fma2(scale.v[i][j], u, x[i].pair(j));
        if constexpr (PRE) q = fma2(o[i][j], o[i][j], q);
        w.set(j, o[i][j]);
      }
      const int c = (i * a.tpr + lane) * V;
      if (mine && c < a.n && a.out) w.store(static_cast<T*>(a.out) + row * a.n + c);
    }
    if constexpr (PRE) {
      float ss[1] = {q.x + q.y};
      row_sum<1, NARROW>(ss, a.tpr, sm, turn);
      r2 = rsqrtf(fmaf(ss[0], inv, a.eps));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        Piece<T> w;
#pragma unroll
        for (int j = 0; j < P; ++j) w.set(j, mul2(mul2(o[i][j], both(r2)), pre.v[i][j]));
        const int c = (i * a.tpr + lane) * V;
        if (mine && c < a.n) w.store(static_cast<T*>(a.normed) + row * a.n + c);
      }
    }
    if (a.stats && mine && lane == 0) *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(r1, r2);
  }
  copy_wait<0>();
}

// A CTA's parameter sums, kept by its threads, to its part of a.partial.
template <int NV, int V, bool NARROW>
__device__ __forceinline__ void put_sums(const NormArgs& a, const float (&sums)[3][NV][V], float* cols, int lane, int sub, int per) {
  float* const mine = a.partial + static_cast<long long>(blockIdx.x) * 3 * a.n;
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    if constexpr (NARROW) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = (i * a.tpr + lane) * V + j;
          if (c < a.n) cols[sub * a.n + c] = sums[p][i][j];
        }
      __syncthreads();
      for (int c = threadIdx.x; c < a.n; c += kNormNarrow) {
        float s = 0.f;
        for (int q = 0; q < per; ++q) s += cols[q * a.n + c];
        mine[p * a.n + c] = s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = (i * a.tpr + lane) * V + j;
          if (c < a.n) mine[p * a.n + c] = sums[p][i][j];
        }
    }
  }
}

template <typename T, int NV, bool NARROW, bool GATE, bool PRE, int S>
__global__ void __launch_bounds__(NARROW ? kNormNarrow : 512, NARROW ? 2 : 1) norm_backward_ring_kernel(NormArgs a) {
  constexpr int V = 16 / sizeof(T), P = V / 2, K = 2 + GATE + 2 * PRE;
  extern __shared__ __align__(16) uint4 ring_places[];
  __shared__ float sm[2][32][4];
  int turn = 0;
  const int lane = NARROW ? static_cast<int>(threadIdx.x) % a.tpr : static_cast<int>(threadIdx.x);
  const int per = NARROW ? kNormNarrow / a.tpr : 1, sub = NARROW ? static_cast<int>(threadIdx.x) / a.tpr : 0;
  const float inv = 1.f / static_cast<float>(a.n);
  const long long step = static_cast<long long>(gridDim.x) * per;
  NormRing<T, NV, K, S> ring{ring_places + threadIdx.x, static_cast<int>(blockDim.x)};
  ring.set(0, a.y, a.y);
  ring.set(1, a.dout, a.y);
  if constexpr (GATE) ring.set(2, a.gate, a.y);
  if constexpr (PRE) {
    ring.set(2 + GATE, a.residual, a.y);
    ring.set(3 + GATE, a.dnormed, a.y);
  }
  long long first = static_cast<long long>(blockIdx.x) * per;
#pragma unroll
  for (int s = 0; s < S; ++s) ring.issue(s, first + s * step + sub, first + s * step + sub < a.rows, lane, a.tpr, a.n);
  auto stats_of = [&](long long row) {
    return a.stats && row < a.rows ? __ldg(reinterpret_cast<const float2*>(a.stats) + row) : both(1.f);
  };
  float2 ahead = stats_of(first + sub);
  Weights<NV, V> post, scale, pre;
  post.load(a.post, lane, a.tpr, a.n);
  scale.load(a.scale, lane, a.tpr, a.n);
  if constexpr (PRE) pre.load(a.pre, lane, a.tpr, a.n);
  float2 sums[3][NV][P];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < P; ++j) sums[0][i][j] = sums[1][i][j] = sums[2][i][j] = both(0.f);

  for (int s = 0; first < a.rows; first += step, s = s + 1 == S ? 0 : s + 1) {
    const long long row = first + sub;
    copy_wait<S - 1>();
    Piece<T> y[NV], po[NV], g[NV], x[NV], pn[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      y[i] = ring.get(s, 0, i);
      po[i] = ring.get(s, 1, i);
      if constexpr (GATE) g[i] = ring.get(s, 2, i);
      if constexpr (PRE) {
        x[i] = ring.get(s, 2 + GATE, i);
        pn[i] = ring.get(s, 3 + GATE, i);
      }
    }
    ring.issue(s, row + S * step, row + S * step < a.rows, lane, a.tpr, a.n);
    const float r1 = ahead.x, r2 = ahead.y;
    ahead = stats_of(row + step);
    float2 act[NV][P], slope[NV][P], u[NV][P], D[NV][P];  // silu(gate), its slope, act post yn, gradient of out
    float2 S1 = both(0.f), S2 = both(0.f), S3 = both(0.f), S4 = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < P; ++j) {
        u[i][j] = mul2(mul2(y[i].pair(j), both(r1)), post.v[i][j]);
        if constexpr (GATE) {
          const float2 f = g[i].pair(j), sg = make_float2(sigmoid(f.x), sigmoid(f.y));
          act[i][j] = mul2(f, sg);
          slope[i][j] = fma2(act[i][j], fma2(sg, both(-1.f), both(1.f)), sg);
          u[i][j] = mul2(act[i][j], u[i][j]);
        }
        const float2 m = mul2(scale.v[i][j], u[i][j]), dout = po[i].pair(j);
        S2 = fma2(m, dout, S2);
        if constexpr (PRE) {
          const float2 out = fma2(scale.v[i][j], u[i][j], x[i].pair(j)), d = mul2(pn[i].pair(j), pre.v[i][j]);
          S1 = fma2(d, out, S1);
          S3 = fma2(m, d, S3);
          S4 = fma2(m, out, S4);
          D[i][j] = out;  // for now
        } else {
          D[i][j] = dout;
        }
      }
    float k = 0.f, ky;  // mean(d on); r1^2 mean(e yn), as dy = r1 e - y ky
    if constexpr (PRE) {
      float v[4] = {S1.x + S1.y, S2.x + S2.y, S3.x + S3.y, S4.x + S4.y};
      row_sum<4, NARROW>(v, a.tpr, sm, turn);
      k = v[0] * inv * r2;
      ky = fmaf(r2, fmaf(-k * r2, v[3], v[2]), v[1]);
    } else {
      float v[1] = {S2.x + S2.y};
      if (a.post) row_sum<1, NARROW>(v, a.tpr, sm, turn);
      ky = v[0];
    }
    ky = a.post ? ky * inv * r1 * r1 : 0.f;
    const bool live_row = row < a.rows;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * a.tpr + lane) * V;
      const bool live = live_row && c < a.n;
      const long long at = row * a.n + c;
      Piece<T> wx, wg, wy;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        if constexpr (PRE) {
          const float2 on = mul2(D[i][j], both(r2)), dn = pn[i].pair(j);
          sums[2][i][j] = fma2(dn, on, sums[2][i][j]);
          D[i][j] = fma2(both(r2), fma2(on, both(-k), mul2(dn, pre.v[i][j])), po[i].pair(j));
        }
        wx.set(j, D[i][j]);
        sums[1][i][j] = fma2(D[i][j], u[i][j], sums[1][i][j]);
        const float2 Ds = mul2(D[i][j], scale.v[i][j]), yn = mul2(y[i].pair(j), both(r1));
        float2 e = Ds;
        if constexpr (GATE) {
          wg.set(j, mul2(mul2(Ds, mul2(yn, post.v[i][j])), slope[i][j]));
          e = mul2(e, act[i][j]);
        }
        sums[0][i][j] = fma2(e, yn, sums[0][i][j]);
        wy.set(j, fma2(y[i].pair(j), both(-ky), mul2(mul2(e, post.v[i][j]), both(r1))));
      }
      if (live && a.dresidual) wx.store(static_cast<T*>(a.dresidual) + at);
      if constexpr (GATE) {
        if (live && a.dgate) wg.store(static_cast<T*>(a.dgate) + at);
      }
      if (live && a.dy) wy.store(static_cast<T*>(a.dy) + at);
    }
  }
  copy_wait<0>();
  if (!a.partial) return;
  float flat[3][NV][V];
#pragma unroll
  for (int p = 0; p < 3; ++p)
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < P; ++j) {
        flat[p][i][2 * j] = sums[p][i][j].x;
        flat[p][i][2 * j + 1] = sums[p][i][j].y;
      }
  put_sums<NV, V, NARROW>(a, flat, reinterpret_cast<float*>(ring_places), lane, sub, per);
}

// -- many wide rows, backward: rows in a pipeline ------------------------------------
//
// A row's sums have to meet across the CTA before its gradients can be formed.  With
// one row at a time every warp waits there.  So row i + 1's sums are formed before
// row i's gradients, both from the ring: what its threads send each other travels
// meanwhile, and one barrier a row is enough.  The second conversion and sigmoid
// cost less than the wait: 16384 x 4096 bf16 267 us one row at a time, 248 us so (the
// same traffic without the arithmetic: 175 us).  The forward pass, interleaved over
// three rows in the same way, went from 132 to 169 us: it stays as it is.

// Sums of K values over a CTA's threads in two halves: send() leaves a warp's in
// shared memory, get() after the barrier adds them up.
template <int K>
struct RowExchange {
  float (*sm)[32][4];
  __device__ __forceinline__ void send(int turn, const float (&v)[K]) const {
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    if constexpr (K == 4) {
      const bool up = lane & 16, odd = lane & 8;
      float a = up ? v[2] : v[0], b = up ? v[3] : v[1];
      a += __shfl_xor_sync(~0u, up ? v[0] : v[2], 16);
      b += __shfl_xor_sync(~0u, up ? v[1] : v[3], 16);
      float c = odd ? b : a;
      c += __shfl_xor_sync(~0u, odd ? a : b, 8);
      c += __shfl_xor_sync(~0u, c, 4);
      c += __shfl_xor_sync(~0u, c, 2);
      c += __shfl_xor_sync(~0u, c, 1);
      if ((lane & 7) == 0) sm[turn][w][lane / 8] = c;
    } else {
      float c = v[0];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(~0u, c, o);
      if (lane == 0) sm[turn][w][0] = c;
    }
  }
  __device__ __forceinline__ void get(int turn, int warps, float (&v)[K]) const {
    const int lane = threadIdx.x % 32;
    float c = 0.f;
    for (int w = lane / K; w < warps; w += 32 / K) c += sm[turn][w][lane % K];
#pragma unroll
    for (int o = K; o < 32; o <<= 1) c += __shfl_xor_sync(~0u, c, o);
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = K == 1 ? c : __shfl_sync(~0u, c, k);
  }
};

// 16 bytes a thread and tensor.
template <typename T, bool GATE, bool PRE>
__global__ void __launch_bounds__(512, 1) norm_backward_pipe_kernel(NormArgs a) {
  constexpr int V = 16 / sizeof(T), P = V / 2, K = 2 + GATE + 2 * PRE, S = 4, KS = PRE ? 4 : 1;
  extern __shared__ __align__(16) uint4 ring_places[];
  __shared__ float sm[2][32][4];
  const int lane = threadIdx.x, c = lane * V, warps = a.tpr / 32;
  const float inv = 1.f / static_cast<float>(a.n);
  NormRing<T, 1, K, S> ring{ring_places + threadIdx.x, static_cast<int>(blockDim.x)};
  ring.set(0, a.y, a.y);
  ring.set(1, a.dout, a.y);
  if constexpr (GATE) ring.set(2, a.gate, a.y);
  if constexpr (PRE) {
    ring.set(2 + GATE, a.residual, a.y);
    ring.set(3 + GATE, a.dnormed, a.y);
  }
  const RowExchange<KS> ex{sm};
  const long long step = gridDim.x;
  const int rows = static_cast<int>((a.rows - blockIdx.x + step - 1) / step);  // of this CTA
  auto row_of = [&](int i) { return blockIdx.x + i * step; };
  auto stats_of = [&](int i) { return a.stats && i < rows ? __ldg(reinterpret_cast<const float2*>(a.stats) + row_of(i)) : both(1.f); };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) ring.issue(s, row_of(s), s < rows, lane, a.tpr, a.n);
  Weights<1, V> post, scale, pre;
  post.load(a.post, lane, a.tpr, a.n);
  scale.load(a.scale, lane, a.tpr, a.n);
  if constexpr (PRE) pre.load(a.pre, lane, a.tpr, a.n);
  float2 sums[3][P];
#pragma unroll
  for (int j = 0; j < P; ++j) sums[0][j] = sums[1][j] = sums[2][j] = both(0.f);
  float2 r = both(1.f), next = stats_of(0), ahead;  // r1, r2 of rows i, i + 1, i + 2
  float k = 0.f, ky = 0.f;                          // of row i: mean(d on); r1^2 mean(e yn), as dy = r1 e - y ky
  for (int i = -1; i < rows; ++i) {
    ahead = stats_of(i + 2);
    copy_wait<S - 2>();  // row i + 1 is here
    float v[KS];
#pragma unroll
    for (int q = 0; q < KS; ++q) v[q] = 0.f;
    if (i + 1 < rows) {
      const int s = (i + 1) & (S - 1);
      const Piece<T> y = ring.get(s, 0, 0), po = ring.get(s, 1, 0);
      Piece<T> g, x, pn;
      if constexpr (GATE) g = ring.get(s, 2, 0);
      if constexpr (PRE) {
        x = ring.get(s, 2 + GATE, 0);
        pn = ring.get(s, 3 + GATE, 0);
      }
      float2 S1 = both(0.f), S2 = both(0.f), S3 = both(0.f), S4 = both(0.f);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        float2 m = mul2(mul2(mul2(y.pair(j), both(next.x)), post.v[0][j]), scale.v[0][j]);
        if constexpr (GATE) {
          const float2 f = g.pair(j);
          m = mul2(mul2(f, make_float2(sigmoid(f.x), sigmoid(f.y))), m);
        }
        S2 = fma2(m, po.pair(j), S2);
        if constexpr (PRE) {
          const float2 out = __fadd2_rn(m, x.pair(j)), d = mul2(pn.pair(j), pre.v[0][j]);
          S1 = fma2(d, out, S1);
          S3 = fma2(m, d, S3);
          S4 = fma2(m, out, S4);
        }
      }
      if constexpr (PRE) {
        v[0] = S1.x + S1.y;
        v[1] = S2.x + S2.y;
        v[2] = S3.x + S3.y;
        v[3] = S4.x + S4.y;
      } else {
        v[0] = S2.x + S2.y;
      }
    }
    const int turn = i & 1;
    ex.send(turn, v);
    if (i >= 0) {
      const int s = i & (S - 1);
      const Piece<T> y = ring.get(s, 0, 0), po = ring.get(s, 1, 0);
      Piece<T> g, x, pn, wx, wg, wy;
      if constexpr (GATE) g = ring.get(s, 2, 0);
      if constexpr (PRE) {
        x = ring.get(s, 2 + GATE, 0);
        pn = ring.get(s, 3 + GATE, 0);
      }
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const float2 yn = mul2(y.pair(j), both(r.x)), t = mul2(yn, post.v[0][j]);
        float2 act, sg, u = t;
        if constexpr (GATE) {
          const float2 f = g.pair(j);
          sg = make_float2(sigmoid(f.x), sigmoid(f.y));
          act = mul2(f, sg);
          u = mul2(act, t);
        }
        float2 D = po.pair(j);  // gradient of out
        if constexpr (PRE) {
          const float2 on = mul2(fma2(scale.v[0][j], u, x.pair(j)), both(r.y)), dn = pn.pair(j);
          sums[2][j] = fma2(dn, on, sums[2][j]);
          D = fma2(both(r.y), fma2(on, both(-k), mul2(dn, pre.v[0][j])), D);
        }
        wx.set(j, D);
        sums[1][j] = fma2(D, u, sums[1][j]);
        float2 e = mul2(D, scale.v[0][j]);
        if constexpr (GATE) {
          wg.set(j, mul2(mul2(e, t), fma2(act, fma2(sg, both(-1.f), both(1.f)), sg)));
          e = mul2(e, act);
        }
        sums[0][j] = fma2(e, yn, sums[0][j]);
        wy.set(j, fma2(y.pair(j), both(-ky), mul2(mul2(e, post.v[0][j]), both(r.x))));
      }
      const long long at = row_of(i) * a.n + c;
      if (c < a.n) {
        if (a.dresidual) wx.store(static_cast<T*>(a.dresidual) + at);
        if constexpr (GATE) {
          if (a.dgate) wg.store(static_cast<T*>(a.dgate) + at);
        }
        if (a.dy) wy.store(static_cast<T*>(a.dy) + at);
      }
    }
    ring.issue((i + S) & (S - 1), row_of(i + S), i + S < rows, lane, a.tpr, a.n);  // row i's places
    __syncthreads();
    ex.get(turn, warps, v);
    r = next;
    next = ahead;
    if constexpr (PRE) {
      k = v[0] * inv * r.y;
      ky = fmaf(r.y, fmaf(-k * r.y, v[3], v[2]), v[1]);
    } else {
      ky = v[0];
    }
    ky = a.post ? ky * inv * r.x * r.x : 0.f;
  }
  copy_wait<0>();
  if (!a.partial) return;
  float flat[3][1][V];
#pragma unroll
  for (int p = 0; p < 3; ++p)
#pragma unroll
    for (int j = 0; j < P; ++j) {
      flat[p][0][2 * j] = sums[p][j].x;
      flat[p][0][2 * j + 1] = sums[p][j].y;
    }
  put_sums<1, V, false>(a, flat, nullptr, lane, 0, 1);
}

// -- rows on any address -------------------------------------------------------------

template <typename T>
__device__ __forceinline__ float load_or_zero(const void* p, long long at, bool live) {
  return live && p ? to_f32(static_cast<const T*>(p)[at]) : 0.f;
}

__device__ __forceinline__ float load_weight(const float* p, int c, bool live) { return live && p ? __ldg(p + c) : 1.f; }

// One channel a thread and step, NV steps.
template <typename T, int NV, bool NARROW>
__global__ void __launch_bounds__(NARROW ? kNormNarrow : 1024, NARROW || NV > 2 ? 1 : 2) norm_kernel(NormArgs a) {
  __shared__ float sm[2][32][4];
  int turn = 0;
  const int lane = NARROW ? static_cast<int>(threadIdx.x) % a.tpr : static_cast<int>(threadIdx.x);
  const long long row = NARROW ? static_cast<long long>(blockIdx.x) * (kNormNarrow / a.tpr) + threadIdx.x / a.tpr
                               : static_cast<long long>(blockIdx.x);
  const bool here = row < a.rows && wanted(a, row);
  const float inv = 1.f / static_cast<float>(a.n);
  float y[NV], g[NV], o[NV], ss[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * a.tpr + lane;
    const bool live = here && c < a.n;
    y[i] = load_or_zero<T>(a.y, row * a.n + c, live);
    g[i] = load_or_zero<T>(a.gate, row * a.n + c, live);
    o[i] = load_or_zero<T>(a.residual, row * a.n + c, live);
    ss[0] = fmaf(y[i], y[i], ss[0]);
  }
  float r1 = 1.f;
  if (a.post) {
    row_sum<1, NARROW>(ss, a.tpr, sm, turn);
    r1 = rsqrtf(fmaf(ss[0], inv, a.eps));
  }
  ss[0] = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * a.tpr + lane;
    const bool live = here && c < a.n;
    float u = y[i] * r1 * load_weight(a.post, c, live);
    if (a.gate) u *= g[i] * sigmoid(g[i]);
    o[i] = fmaf(load_weight(a.scale, c, live), u, o[i]);
    ss[0] = fmaf(o[i], o[i], ss[0]);
    if (live && a.out) static_cast<T*>(a.out)[row * a.n + c] = from_f32<T>(o[i]);
  }
  float r2 = 1.f;
  if (a.pre) {
    row_sum<1, NARROW>(ss, a.tpr, sm, turn);
    r2 = rsqrtf(fmaf(ss[0], inv, a.eps));
  }
  if (a.stats && here && lane == 0) *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(r1, r2);
  if (!a.pre) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * a.tpr + lane;
    if (here && c < a.n) static_cast<T*>(a.normed)[row * a.n + c] = from_f32<T>(o[i] * r2 * load_weight(a.pre, c, true));
  }
}

// A CTA takes every gridDim.x-th row (narrow: 256 / tpr rows at a time).
template <typename T, int NV, bool NARROW>
__global__ void __launch_bounds__(NARROW ? kNormNarrow : 1024, NARROW || NV > 2 ? 1 : 2) norm_backward_kernel(NormArgs a) {
  __shared__ float sm[2][32][4];
  extern __shared__ float cols[];  // narrow: [256 / tpr][n] of one parameter at a time
  int turn = 0;
  const int lane = NARROW ? static_cast<int>(threadIdx.x) % a.tpr : static_cast<int>(threadIdx.x);
  const int per = NARROW ? kNormNarrow / a.tpr : 1, sub = NARROW ? static_cast<int>(threadIdx.x) / a.tpr : 0;
  const float inv = 1.f / static_cast<float>(a.n);
  float sums[3][NV][1];
#pragma unroll
  for (int i = 0; i < NV; ++i) sums[0][i][0] = sums[1][i][0] = sums[2][i][0] = 0.f;

  for (long long first = static_cast<long long>(blockIdx.x) * per; first < a.rows; first += static_cast<long long>(gridDim.x) * per) {
    const long long row = first + sub;
    float y[NV], g[NV], D[NV], pn[NV], x[NV], v[4] = {0.f, 0.f, 0.f, 0.f};  // v: S1 to S4
    const float2 r = a.stats && row < a.rows ? __ldg(reinterpret_cast<const float2*>(a.stats) + row) : make_float2(1.f, 1.f);
    const float r1 = r.x, r2 = r.y;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * a.tpr + lane;
      const bool live = row < a.rows && c < a.n;
      y[i] = load_or_zero<T>(a.y, row * a.n + c, live);
      g[i] = load_or_zero<T>(a.gate, row * a.n + c, live);
      D[i] = load_or_zero<T>(a.dout, row * a.n + c, live);
      x[i] = load_or_zero<T>(a.pre ? a.residual : nullptr, row * a.n + c, live);
      pn[i] = load_or_zero<T>(a.pre ? a.dnormed : nullptr, row * a.n + c, live);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * a.tpr + lane;
      const bool live = row < a.rows && c < a.n;
      const float scale = load_weight(a.scale, c, live), d = pn[i] * load_weight(a.pre, c, live);
      float u = y[i] * r1 * load_weight(a.post, c, live);
      if (a.gate) u *= g[i] * sigmoid(g[i]);
      x[i] = fmaf(scale, u, x[i]);  // out from here on
      u *= scale;
      v[0] = fmaf(d, x[i], v[0]);
      v[1] = fmaf(u, D[i], v[1]);
      v[2] = fmaf(u, d, v[2]);
      v[3] = fmaf(u, x[i], v[3]);
    }
    if (a.post || a.pre) row_sum<4, NARROW>(v, a.tpr, sm, turn);
    const float k = a.pre ? v[0] * inv * r2 : 0.f;  // mean(d on)
    const float ky = a.post ? (a.pre ? fmaf(r2, fmaf(-k * r2, v[3], v[2]), v[1]) : v[1]) * inv * r1 * r1 : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * a.tpr + lane;
      const bool live = row < a.rows && c < a.n;
      const float post = load_weight(a.post, c, live), scale = load_weight(a.scale, c, live), yn = y[i] * r1;
      if (a.pre) {
        const float on = x[i] * r2;
        sums[2][i][0] = fmaf(pn[i], on, sums[2][i][0]);
        D[i] = fmaf(r2, pn[i] * load_weight(a.pre, c, live) - on * k, D[i]);
      }
      float act = 1.f, slope = 0.f;
      if (a.gate) {
        const float sg = sigmoid(g[i]);
        act = g[i] * sg;
        slope = fmaf(act, 1.f - sg, sg);
      }
      const float Ds = D[i] * scale, t = post * yn;
      sums[0][i][0] = fmaf(Ds * act, yn, sums[0][i][0]);
      sums[1][i][0] = fmaf(D[i] * act, t, sums[1][i][0]);
      if (live && a.dresidual) static_cast<T*>(a.dresidual)[row * a.n + c] = from_f32<T>(D[i]);
      if (live && a.dgate) static_cast<T*>(a.dgate)[row * a.n + c] = from_f32<T>(Ds * t * slope);
      if (live && a.dy) static_cast<T*>(a.dy)[row * a.n + c] = from_f32<T>(fmaf(y[i], -ky, Ds * act * post * r1));
    }
  }
  if (a.partial) put_sums<NV, 1, NARROW>(a, sums, cols, lane, sub, per);
}

// -- many rows on any address of tensors that start on 16 bytes -------------------------
//
// CTAs stay.  The aligned 16-byte units that cover a group's next row travel by
// cp.async into its places in shared memory, [2][tensors][units], while this row is
// worked on, and are read at the row's own shift; weights stay in registers.  The
// arithmetic is that of the kernels above: with both forms in one template, those
// lost 10 to 50% to registers they have not got.
template <typename T, bool NARROW>
struct AheadRows {
  unsigned char* mine;  // this group's places
  int tensors, units, lane, tpr, n;
  long long bytes;      // of a tensor
  int stage = 0;

  __device__ __forceinline__ AheadRows(const NormArgs& a, unsigned char* ring, int tensors, int sub, int lane, int tpr)
      : tensors(tensors), units(ahead_units<T>(a.n)), lane(lane), tpr(tpr), n(a.n), bytes(a.rows * a.n * static_cast<long long>(sizeof(T))) {
    mine = ring + static_cast<long long>(sub) * 2 * tensors * units * 16;
  }
  __device__ __forceinline__ unsigned char* place(int st, int k) const { return mine + (st * tensors + k) * units * 16; }
  __device__ __forceinline__ void fetch(int st, int k, const void* p, long long row) const {
    const long long from = row * n * static_cast<long long>(sizeof(T)), at = from & ~15ll;
    const int need = static_cast<int>(from - at) + n * static_cast<int>(sizeof(T));
    for (int u = lane; u * 16 < need; u += tpr) {
      const long long left = bytes - at - 16 * u;  // of the tensor, at least 1
      copy_async16(place(st, k) + u * 16, static_cast<const unsigned char*>(p) + at + 16 * u, left < 16 ? static_cast<int>(left) : 16);
    }
  }
  // Everything that fetch() was called for is there, for the whole group.
  __device__ __forceinline__ void turn() {
    copy_wait<0>();
    if constexpr (NARROW) __syncwarp();
    else __syncthreads();
  }
  __device__ __forceinline__ float get(int k, const void* p, long long row, int c, bool live) const {
    if (!live || !p) return 0.f;
    const int shift = static_cast<int>(static_cast<unsigned>(row) * static_cast<unsigned>(n) % (16 / sizeof(T)));
    return to_f32(reinterpret_cast<const T*>(place(stage, k))[shift + c]);
  }
};

// A thread's channels of a weight vector.
template <int NV>
struct AheadWeight {
  float w[NV];
  __device__ __forceinline__ AheadWeight(const float* p, int n, int tpr, int lane) {
#pragma unroll
    for (int i = 0; i < NV; ++i) w[i] = load_weight(p, i * tpr + lane, i * tpr + lane < n);
  }
};

// Narrow: a warp a row.
template <typename T, int NV, bool NARROW>
__global__ void __launch_bounds__(NARROW ? kNormNarrow : 512, NARROW ? 3 : 2) norm_ahead_kernel(NormArgs a) {
  __shared__ float sm[2][32][4];
  extern __shared__ __align__(16) unsigned char ahead_places[];
  int turn = 0;
  const int tpr = NARROW ? 32 : a.tpr;
  const int lane = NARROW ? static_cast<int>(threadIdx.x) % tpr : static_cast<int>(threadIdx.x);
  const int per = NARROW ? kNormNarrow / tpr : 1, sub = NARROW ? static_cast<int>(threadIdx.x) / tpr : 0;
  const float inv = 1.f / static_cast<float>(a.n);
  const int kg = 1, kr = kg + (a.gate != nullptr);
  AheadRows<T, NARROW> in(a, ahead_places, kr + (a.residual != nullptr), sub, lane, tpr);
  const AheadWeight<NV> post(a.post, a.n, tpr, lane), scale(a.scale, a.n, tpr, lane), pre(a.pre, a.n, tpr, lane);
  auto fetch = [&](int st, long long row) {
    if (row < a.rows) {
      in.fetch(st, 0, a.y, row);
      if (a.gate) in.fetch(st, kg, a.gate, row);
      if (a.residual) in.fetch(st, kr, a.residual, row);
    }
    copy_commit();
  };
  const long long step = static_cast<long long>(gridDim.x) * per;
  fetch(0, static_cast<long long>(blockIdx.x) * per + sub);
  for (long long first = static_cast<long long>(blockIdx.x) * per; first < a.rows; first += step) {
    const long long row = first + sub;
    const bool here = row < a.rows && wanted(a, row);
    in.turn();
    fetch(in.stage ^ 1, row + step);
    float y[NV], g[NV], o[NV], ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * tpr + lane;
      const bool live = here && c < a.n;
      y[i] = in.get(0, a.y, row, c, live);
      g[i] = in.get(kg, a.gate, row, c, live);
      o[i] = in.get(kr, a.residual, row, c, live);
      ss[0] = fmaf(y[i], y[i], ss[0]);
    }
    float r1 = 1.f;
    if (a.post) {
      row_sum<1, NARROW>(ss, tpr, sm, turn);
      r1 = rsqrtf(fmaf(ss[0], inv, a.eps));
    }
    ss[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * tpr + lane;
      const bool live = here && c < a.n;
      float u = y[i] * r1 * post.w[i];
      if (a.gate) u *= g[i] * sigmoid(g[i]);
      o[i] = fmaf(scale.w[i], u, o[i]);
      ss[0] = fmaf(o[i], o[i], ss[0]);
      if (live && a.out) static_cast<T*>(a.out)[row * a.n + c] = from_f32<T>(o[i]);
    }
    float r2 = 1.f;
    if (a.pre) {
      row_sum<1, NARROW>(ss, tpr, sm, turn);
      r2 = rsqrtf(fmaf(ss[0], inv, a.eps));
    }
    if (a.stats && here && lane == 0) *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(r1, r2);
    in.stage ^= 1;
    if (!a.pre) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * tpr + lane;
      if (here && c < a.n) static_cast<T*>(a.normed)[row * a.n + c] = from_f32<T>(o[i] * r2 * pre.w[i]);
    }
  }
}

template <typename T, int NV, bool NARROW>
__global__ void __launch_bounds__(NARROW ? kNormNarrow : 512, NARROW ? 2 : 1) norm_backward_ahead_kernel(NormArgs a) {
  __shared__ float sm[2][32][4];
  extern __shared__ __align__(16) unsigned char ahead_places[];
  float* const cols = reinterpret_cast<float*>(ahead_places);  // after the rows; narrow: [256 / tpr][n] of one parameter at a time
  int turn = 0;
  const int tpr = NARROW ? 32 : a.tpr;
  const int lane = NARROW ? static_cast<int>(threadIdx.x) % tpr : static_cast<int>(threadIdx.x);
  const int per = NARROW ? kNormNarrow / tpr : 1, sub = NARROW ? static_cast<int>(threadIdx.x) / tpr : 0;
  const float inv = 1.f / static_cast<float>(a.n);
  float sums[3][NV][1];
#pragma unroll
  for (int i = 0; i < NV; ++i) sums[0][i][0] = sums[1][i][0] = sums[2][i][0] = 0.f;

  const void* const residual = a.pre ? a.residual : nullptr;
  const int kg = 1, kd = kg + (a.gate != nullptr), kr = kd + (a.dout != nullptr), kp = kr + (residual != nullptr);
  AheadRows<T, NARROW> in(a, ahead_places, kp + (a.dnormed != nullptr), sub, lane, tpr);
  const AheadWeight<NV> wpost(a.post, a.n, tpr, lane), wscale(a.scale, a.n, tpr, lane), wpre(a.pre, a.n, tpr, lane);
  auto fetch = [&](int st, long long row) {
    if (row < a.rows) {
      in.fetch(st, 0, a.y, row);
      if (a.gate) in.fetch(st, kg, a.gate, row);
      if (a.dout) in.fetch(st, kd, a.dout, row);
      if (residual) in.fetch(st, kr, residual, row);
      if (a.dnormed) in.fetch(st, kp, a.dnormed, row);
    }
    copy_commit();
  };
  const long long step = static_cast<long long>(gridDim.x) * per;
  fetch(0, static_cast<long long>(blockIdx.x) * per + sub);
  for (long long first = static_cast<long long>(blockIdx.x) * per; first < a.rows; first += step) {
    const long long row = first + sub;
    in.turn();
    fetch(in.stage ^ 1, row + step);
    float y[NV], g[NV], D[NV], pn[NV], x[NV], v[4] = {0.f, 0.f, 0.f, 0.f};  // v: S1 to S4
    const float2 r = a.stats && row < a.rows ? __ldg(reinterpret_cast<const float2*>(a.stats) + row) : make_float2(1.f, 1.f);
    const float r1 = r.x, r2 = r.y;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * tpr + lane;
      const bool live = row < a.rows && c < a.n;
      y[i] = in.get(0, a.y, row, c, live);
      g[i] = in.get(kg, a.gate, row, c, live);
      D[i] = in.get(kd, a.dout, row, c, live);
      x[i] = in.get(kr, residual, row, c, live);
      pn[i] = in.get(kp, a.dnormed, row, c, live);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float scale = wscale.w[i], d = pn[i] * wpre.w[i];
      float u = y[i] * r1 * wpost.w[i];
      if (a.gate) u *= g[i] * sigmoid(g[i]);
      x[i] = fmaf(scale, u, x[i]);  // out from here on
      u *= scale;
      v[0] = fmaf(d, x[i], v[0]);
      v[1] = fmaf(u, D[i], v[1]);
      v[2] = fmaf(u, d, v[2]);
      v[3] = fmaf(u, x[i], v[3]);
    }
    if (a.post || a.pre) row_sum<4, NARROW>(v, tpr, sm, turn);
    const float k = a.pre ? v[0] * inv * r2 : 0.f;  // mean(d on)
    const float ky = a.post ? (a.pre ? fmaf(r2, fmaf(-k * r2, v[3], v[2]), v[1]) : v[1]) * inv * r1 * r1 : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * tpr + lane;
      const bool live = row < a.rows && c < a.n;
      const float post = wpost.w[i], scale = wscale.w[i], yn = y[i] * r1;
      if (a.pre) {
        const float on = x[i] * r2;
        sums[2][i][0] = fmaf(pn[i], on, sums[2][i][0]);
        D[i] = fmaf(r2, pn[i] * wpre.w[i] - on * k, D[i]);
      }
      float act = 1.f, slope = 0.f;
      if (a.gate) {
        const float sg = sigmoid(g[i]);
        act = g[i] * sg;
        slope = fmaf(act, 1.f - sg, sg);
      }
      const float Ds = D[i] * scale, t = post * yn;
      sums[0][i][0] = fmaf(Ds * act, yn, sums[0][i][0]);
      sums[1][i][0] = fmaf(D[i] * act, t, sums[1][i][0]);
      if (live && a.dresidual) static_cast<T*>(a.dresidual)[row * a.n + c] = from_f32<T>(D[i]);
      if (live && a.dgate) static_cast<T*>(a.dgate)[row * a.n + c] = from_f32<T>(Ds * t * slope);
      if (live && a.dy) static_cast<T*>(a.dy)[row * a.n + c] = from_f32<T>(fmaf(y[i], -ky, Ds * act * post * r1));
    }
    in.stage ^= 1;
  }
  if (a.partial) put_sums<NV, 1, NARROW>(a, sums, cols, lane, sub, per);
}

// Parameter gradients from the CTAs' sums: grid (columns / 32, 3), 32 x 32 threads.
__global__ void __launch_bounds__(1024) norm_sums_kernel(const float* partial, int ctas, int n, float* dpost, float* dscale, float* dpre) {
  __shared__ float sm[32][33];
  float* const to = blockIdx.y == 0 ? dpost : blockIdx.y == 1 ? dscale : dpre;
  if (!to) return;
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < n)
    for (int q = threadIdx.y; q < ctas; q += 32) s += partial[(static_cast<long long>(q) * 3 + blockIdx.y) * n + c];
  sm[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = sm[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  const int col = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && col < n) to[col] = s;
}

}  // namespace dl
