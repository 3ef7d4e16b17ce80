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
// rounded to its type, and reading residual costs what reading out would.
//
// Bound: memory (10 bytes an element forward, 16 backward in bf16, against
// some 15 and 40 flops).  A row lies in the registers of one group of threads,
// so it is read once; weights come from the L1 cache.  Narrow rows (heads)
// share a CTA, 8 to 32 threads a row; wide rows take a CTA each.
#pragma once

#include "ops.cuh"

namespace dl {

constexpr int kNormMax = 8192;  // channels of a row
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
  float* partial;        // [CTAs][3][n]: post, scale, pre sums of the CTA's rows, or null
  const int* slot_idx;   // [rows / groups] or null: rows to skip
  int slots;
  int groups;            // rows here per row of the slot map
  int n;
  int tpr;               // threads of a row
  long long rows;
  float eps;
};

// Sums K values over the threads of a row.  Narrow: `tpr` (8, 16 or 32) lanes.
// Wide: the whole CTA, through `sm` [2][32][K], whose halves alternate between
// calls so that one barrier a call is enough.
template <int K, bool NARROW>
__device__ __forceinline__ void row_sum(float (&v)[K], int tpr, float (*sm)[32][2], int& turn) {
  if constexpr (NARROW) {
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
    float(*s)[2] = sm[turn];
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

__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + expf(-x)); }

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_or_zero(const void* p, long long at, bool live) {
  if (live && p) return load_stream<T, V>(static_cast<const T*>(p) + at);
  Pack<T, V> z;
#pragma unroll
  for (int j = 0; j < V; ++j) z.v[j] = from_f32<T>(0.f);
  return z;
}

template <int V>
__device__ __forceinline__ Pack<float, V> load_weight(const float* p, int c, bool live) {
  Pack<float, V> w;
#pragma unroll
  for (int j = 0; j < V; ++j) w.v[j] = 1.f;
  if (live && p) {
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(p + c + j));
        w.v[j] = f.x;
        w.v[j + 1] = f.y;
        w.v[j + 2] = f.z;
        w.v[j + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) w.v[j] = __ldg(p + c + j);
    }
  }
  return w;
}

// V channels a load, NV loads a thread and tensor; grid over rows (narrow: 256 / tpr rows a CTA).
template <typename T, int V, int NV, bool NARROW>
__global__ void __launch_bounds__(NARROW ? kNormNarrow : NV == 8 ? 1024 : 512) norm_kernel(NormArgs a) {
  __shared__ float sm[2][32][2];
  int turn = 0;
  const int lane = NARROW ? static_cast<int>(threadIdx.x) % a.tpr : static_cast<int>(threadIdx.x);
  const long long row = NARROW ? static_cast<long long>(blockIdx.x) * (kNormNarrow / a.tpr) + threadIdx.x / a.tpr
                               : static_cast<long long>(blockIdx.x);
  const bool here = row < a.rows && row_slot(a.slot_idx, a.slots, static_cast<int>(row / a.groups), nullptr, false) >= 0;
  const float inv = 1.f / static_cast<float>(a.n);
  Pack<T, V> y[NV], g[NV], x[NV];
  bool live[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * a.tpr + lane) * V;
    live[i] = here && c < a.n;
    y[i] = load_or_zero<T, V>(a.y, row * a.n + c, live[i]);
    g[i] = load_or_zero<T, V>(a.gate, row * a.n + c, live[i]);
    x[i] = load_or_zero<T, V>(a.residual, row * a.n + c, live[i]);
  }
  float r1 = 1.f;
  if (a.post) {
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float f = to_f32(y[i].v[j]);
        ss[0] = fmaf(f, f, ss[0]);
      }
    row_sum<1, NARROW>(ss, a.tpr, sm, turn);
    r1 = rsqrtf(ss[0] * inv + a.eps);
  }
  float o[NV][V];
  float ss[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * a.tpr + lane) * V;
    const Pack<float, V> post = load_weight<V>(a.post, c, live[i]), scale = load_weight<V>(a.scale, c, live[i]);
    Pack<T, V> w;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float u = to_f32(y[i].v[j]) * r1 * post.v[j];
      if (a.gate) {
        const float q = to_f32(g[i].v[j]);
        u *= q * sigmoid(q);
      }
      o[i][j] = fmaf(scale.v[j], u, to_f32(x[i].v[j]));
      ss[0] = fmaf(o[i][j], o[i][j], ss[0]);
      w.v[j] = from_f32<T>(o[i][j]);
    }
    if (live[i] && a.out) store_stream<T, V>(static_cast<T*>(a.out) + row * a.n + c, w);
  }
  if (!a.pre) return;
  row_sum<1, NARROW>(ss, a.tpr, sm, turn);
  const float r2 = rsqrtf(ss[0] * inv + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * a.tpr + lane) * V;
    const Pack<float, V> pre = load_weight<V>(a.pre, c, live[i]);
    Pack<T, V> w;
#pragma unroll
    for (int j = 0; j < V; ++j) w.v[j] = from_f32<T>(o[i][j] * r2 * pre.v[j]);
    if (live[i]) store_stream<T, V>(static_cast<T*>(a.normed) + row * a.n + c, w);
  }
}

// A CTA takes every gridDim.x-th row (narrow: 256 / tpr rows at a time) and
// keeps the parameter sums of its columns in registers; they end in `partial`,
// which norm_sums_kernel adds over the CTAs in order.
template <typename T, int V, int NV, bool NARROW>
__global__ void __launch_bounds__(NARROW ? kNormNarrow : NV == 8 ? 1024 : 512) norm_backward_kernel(NormArgs a) {
  __shared__ float sm[2][32][2];
  extern __shared__ float cols[];  // narrow: [256 / tpr][n] of one parameter at a time
  int turn = 0;
  const int lane = NARROW ? static_cast<int>(threadIdx.x) % a.tpr : static_cast<int>(threadIdx.x);
  const int per = NARROW ? kNormNarrow / a.tpr : 1, sub = NARROW ? static_cast<int>(threadIdx.x) / a.tpr : 0;
  const float inv = 1.f / static_cast<float>(a.n);
  float sums[3][NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) sums[0][i][j] = sums[1][i][j] = sums[2][i][j] = 0.f;

  for (long long first = static_cast<long long>(blockIdx.x) * per; first < a.rows; first += static_cast<long long>(gridDim.x) * per) {
    const long long row = first + sub;
    Pack<T, V> y[NV], g[NV], x[NV], po[NV], pn[NV];
    bool live[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * a.tpr + lane) * V;
      live[i] = row < a.rows && c < a.n;
      y[i] = load_or_zero<T, V>(a.y, row * a.n + c, live[i]);
      g[i] = load_or_zero<T, V>(a.gate, row * a.n + c, live[i]);
      x[i] = load_or_zero<T, V>(a.pre ? a.residual : nullptr, row * a.n + c, live[i]);
      po[i] = load_or_zero<T, V>(a.dout, row * a.n + c, live[i]);
      pn[i] = load_or_zero<T, V>(a.pre ? a.dnormed : nullptr, row * a.n + c, live[i]);
    }
    float r1 = 1.f;
    if (a.post) {
      float ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float f = to_f32(y[i].v[j]);
          ss[0] = fmaf(f, f, ss[0]);
        }
      row_sum<1, NARROW>(ss, a.tpr, sm, turn);
      r1 = rsqrtf(ss[0] * inv + a.eps);
    }
    float D[NV][V];  // gradient of out
    if (a.pre) {
      float ss[2] = {0.f, 0.f};  // out^2, d out
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * a.tpr + lane) * V;
        const Pack<float, V> post = load_weight<V>(a.post, c, live[i]), scale = load_weight<V>(a.scale, c, live[i]),
                             pre = load_weight<V>(a.pre, c, live[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float u = to_f32(y[i].v[j]) * r1 * post.v[j];
          if (a.gate) {
            const float q = to_f32(g[i].v[j]);
            u *= q * sigmoid(q);
          }
          D[i][j] = fmaf(scale.v[j], u, to_f32(x[i].v[j]));  // out for now
          ss[0] = fmaf(D[i][j], D[i][j], ss[0]);
          ss[1] = fmaf(to_f32(pn[i].v[j]) * pre.v[j], D[i][j], ss[1]);
        }
      }
      row_sum<2, NARROW>(ss, a.tpr, sm, turn);
      const float r2 = rsqrtf(ss[0] * inv + a.eps), k = ss[1] * inv * r2;  // k = mean(d on)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const Pack<float, V> pre = load_weight<V>(a.pre, (i * a.tpr + lane) * V, live[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float on = D[i][j] * r2, dn = to_f32(pn[i].v[j]);
          sums[2][i][j] = fmaf(dn, on, sums[2][i][j]);
          D[i][j] = to_f32(po[i].v[j]) + r2 * (dn * pre.v[j] - on * k);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) D[i][j] = to_f32(po[i].v[j]);
    }
    float se[1] = {0.f};  // e yn
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * a.tpr + lane) * V;
      const long long at = row * a.n + c;
      const Pack<float, V> post = load_weight<V>(a.post, c, live[i]), scale = load_weight<V>(a.scale, c, live[i]);
      Pack<T, V> wg, wx;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float yn = to_f32(y[i].v[j]) * r1;
        float act = 1.f, slope = 0.f;
        if (a.gate) {
          const float q = to_f32(g[i].v[j]), sg = sigmoid(q);
          act = q * sg;
          slope = fmaf(act, 1.f - sg, sg);
        }
        wx.v[j] = from_f32<T>(D[i][j]);
        const float Dy = D[i][j] * yn, Ds = D[i][j] * scale.v[j];
        sums[0][i][j] = fmaf(Dy * scale.v[j], act, sums[0][i][j]);
        sums[1][i][j] = fmaf(Dy * post.v[j], act, sums[1][i][j]);
        wg.v[j] = from_f32<T>(Ds * post.v[j] * yn * slope);
        D[i][j] = Ds * post.v[j] * act;  // e
        se[0] = fmaf(D[i][j], yn, se[0]);
      }
      if (live[i] && a.dresidual) store_stream<T, V>(static_cast<T*>(a.dresidual) + at, wx);
      if (live[i] && a.dgate) store_stream<T, V>(static_cast<T*>(a.dgate) + at, wg);
    }
    if (a.dy) {
      float k = 0.f;
      if (a.post) {
        row_sum<1, NARROW>(se, a.tpr, sm, turn);
        k = se[0] * inv;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        Pack<T, V> w;
#pragma unroll
        for (int j = 0; j < V; ++j) w.v[j] = from_f32<T>(r1 * (D[i][j] - to_f32(y[i].v[j]) * r1 * k));
        if (live[i]) store_stream<T, V>(static_cast<T*>(a.dy) + row * a.n + (i * a.tpr + lane) * V, w);
      }
    }
  }
  if (!a.partial) return;
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
