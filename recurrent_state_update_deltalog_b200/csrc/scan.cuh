// Gated linear recurrence h_t = a_t h_{t-1} + x_t, a_t = exp(log_decay_t), per
// channel over packed sequences; its backward pass; its single-token step.
//
// Two steps of the recurrence compose: a run of tokens maps the state before
// it to the state after it as h -> A h + b, with A the product of its a_t and
// b its result from a zero state.  So a sequence is cut into runs, each run
// is reduced to its (A, b) in registers, the pairs are folded in order, and a
// second pass over the same registers produces every h_t from the true state
// before the run.  The inputs are read once.
//
// Bound: memory (2 flops for 8 bytes an element with bf16 x and h).  Layout: a
// CTA of 8 warps holds a chunk of 64 tokens by 32 * V channels, 8 tokens a
// warp, V neighbouring channels a lane, all loads of a chunk in flight at
// once.  Chunks of one sequence run in the CTAs of a cluster side by side: the
// warps of a CTA exchange their (A, b) through shared memory, the CTAs of the
// cluster through distributed shared memory, and the cluster then walks the
// sequence N chunks at a time with the running state in registers.  No global
// flags, no atomics: results do not depend on the order in which CTAs run.
#pragma once

#include "ops.cuh"

namespace dl {

constexpr int kScanWarps = 8;                      // warps of a CTA, consecutive in time
constexpr int kScanTok = 8;                        // tokens a warp holds in registers
constexpr int kScanChunk = kScanWarps * kScanTok;  // tokens of a CTA
static_assert(kScanChunk == DL_SCAN_CHUNK, "checkpoint interval of the interface");

struct ScanArgs {
  const void* x;           // [total][C], TX
  const float* log_decay;  // [total][C]
  const float* h0;         // [slots][C] or null
  float* h_last;           // [slots][C] or null
  void* h;                 // [total][C], TX
  float* ckpt;             // [total / chunk + rows][C] or null: state before each chunk
  const int* slot_idx;     // [rows] or null
  const int* cu;           // [rows + 1] or null: `len` tokens a row
  const void* dh;          // backward: [total][C], TX
  const float* dh_last;    // [rows][C] or null
  void* dx;                // [total][C], TX
  float* dlog_decay;       // [total][C]
  float* dh0;              // [rows][C] or null
  int* err;                // device error word or null
  long long total;
  long long len;           // tokens of every row without cu
  int slots;
  int C;
};

// Tokens of row r; false (row skipped, error raised by one thread) for a range
// outside [0, total].
__device__ __forceinline__ bool scan_row(const ScanArgs& a, int r, bool tell, long long* t0, long long* n) {
  if (!a.cu) {
    *t0 = r * a.len;
    *n = a.len;
    return true;
  }
  const int s = __ldg(a.cu + r), e = __ldg(a.cu + r + 1);
  *t0 = s;
  *n = static_cast<long long>(e) - s;
  if (s < 0 || e < s || e > a.total) {
    if (tell) raise_error(a.err, DL_DEVERR_SEQLEN);
    return false;
  }
  return true;
}

// One warp's tokens [t, t + kScanTok) of a row of n tokens starting at token
// t0, V channels from c, as loaded.  Tokens past the row read as the identity
// (log decay 0, x 0).
template <typename TX, int V>
struct ScanTile {
  Pack<TX, V> x[kScanTok];
  Pack<float, V> d[kScanTok];

  __device__ __forceinline__ void load(const ScanArgs& a, long long t0, long long t, long long n, int c, bool live) {
    const long long base = (t0 + t) * a.C + c;
    const TX* px = static_cast<const TX*>(a.x) + base;
    const float* pd = a.log_decay + base;
#pragma unroll
    for (int i = 0; i < kScanTok; ++i) {
      if (live && t + i < n) {
        x[i] = load_stream<TX, V>(px + static_cast<long long>(i) * a.C);
        d[i] = load_stream<float, V>(pd + static_cast<long long>(i) * a.C);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          x[i].v[j] = from_f32<TX>(0.f);
          d[i].v[j] = 0.f;
        }
      }
    }
  }
};

// Grid (channel tiles * N, rows), clusters of N along x.
template <typename TX, int V, bool CLUSTER>
__global__ void __launch_bounds__(kScanWarps * 32) scan_kernel(ScanArgs a, int N) {
  __shared__ float2 part[2][kScanWarps][32 * V];  // each warp's (A, b)
  __shared__ float2 tot[2][CLUSTER ? 16 : 1][32 * V];

  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
  const int c = (static_cast<int>(blockIdx.x) / N) * (32 * V) + lane * V;
  const int r = blockIdx.y;
  const bool tell = blockIdx.x == 0 && threadIdx.x == 0;
  long long t0, n;
  const int slot = row_slot(a.slot_idx, a.slots, r, a.err, tell);
  if (slot < 0) return;  // the same for every CTA of the cluster
  if (!scan_row(a, r, tell, &t0, &n)) return;
  const bool live = c < a.C;  // C % V == 0

  float carry[V];  // state before the cluster's current N chunks
#pragma unroll
  for (int j = 0; j < V; ++j)
    carry[j] = live && a.h0 ? a.h0[static_cast<long long>(slot) * a.C + c + j] : 0.f;

  ScanTile<TX, V> tile;
  const long long first = static_cast<long long>(rank) * kScanChunk + w * kScanTok;
  const long long stride = static_cast<long long>(N) * kScanChunk;
  const int steps = static_cast<int>((n + stride - 1) / stride);
  if (steps > 0) tile.load(a, t0, first, n, c, live);
  if constexpr (CLUSTER) cluster_sync();  // every CTA of the cluster runs before its shared memory is written
  TX* const out = static_cast<TX*>(a.h);

  for (int s = 0; s < steps; ++s) {
    const long long t = s * stride + first;
    const int buf = s & 1;
    float al[kScanTok][V];
    Pack<TX, V> xs[kScanTok];
    float A[V], b[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      A[j] = 1.f;
      b[j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kScanTok; ++i) {
      xs[i] = tile.x[i];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        al[i][j] = expf(tile.d[i].v[j]);
        b[j] = fmaf(al[i][j], b[j], to_f32(xs[i].v[j]));
        A[j] *= al[i][j];
      }
    }
    if (s + 1 < steps) tile.load(a, t0, t + stride, n, c, live);
#pragma unroll
    for (int j = 0; j < V; ++j) part[buf][w][lane * V + j] = make_float2(A[j], b[j]);
    __syncthreads();

    // (pA, pb): the chunk's warps before this one; the last warp adds its own
    // and hands the chunk's total to every CTA of the cluster
    float pA[V], pb[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      pA[j] = 1.f;
      pb[j] = 0.f;
    }
    for (int i = 0; i < w; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float2 q = part[buf][i][lane * V + j];
        pb[j] = fmaf(q.x, pb[j], q.y);
        pA[j] *= q.x;
      }
    float base[V];  // state before this chunk
    if constexpr (CLUSTER) {
      if (w == kScanWarps - 1) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float tb = fmaf(A[j], pb[j], b[j]), tA = pA[j] * A[j];
          for (int q = 0; q < N; ++q) store_remote(remote_smem(&tot[buf][rank][lane * V + j], q), tA, tb);
        }
      }
      cluster_sync();
#pragma unroll
      for (int j = 0; j < V; ++j) base[j] = carry[j];
      for (int q = 0; q < N; ++q)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (q == rank) base[j] = carry[j];
          const float2 m = tot[buf][q][lane * V + j];
          carry[j] = fmaf(m.x, carry[j], m.y);
        }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) base[j] = carry[j];
      float eA[V], eb[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        eA[j] = pA[j];
        eb[j] = pb[j];
      }
      for (int i = w; i < kScanWarps; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float2 q = part[buf][i][lane * V + j];
          eb[j] = fmaf(q.x, eb[j], q.y);
          eA[j] *= q.x;
        }
#pragma unroll
      for (int j = 0; j < V; ++j) carry[j] = fmaf(eA[j], carry[j], eb[j]);
    }

    if (a.ckpt && w == 0 && live && t < n) {
      const long long row = t0 / kScanChunk + r + t / kScanChunk;
#pragma unroll
      for (int j = 0; j < V; ++j) a.ckpt[row * a.C + c + j] = base[j];
    }
    float hv[V];
#pragma unroll
    for (int j = 0; j < V; ++j) hv[j] = fmaf(pA[j], base[j], pb[j]);
    TX* po = out + (t0 + t) * a.C + c;
#pragma unroll
    for (int i = 0; i < kScanTok; ++i) {
      Pack<TX, V> o;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        hv[j] = fmaf(al[i][j], hv[j], to_f32(xs[i].v[j]));
        o.v[j] = from_f32<TX>(hv[j]);
      }
      if (live && t + i < n) store_stream<TX, V>(po + static_cast<long long>(i) * a.C, o);
    }
  }
  if (a.h_last && live && rank == 0 && w == 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) a.h_last[static_cast<long long>(slot) * a.C + c + j] = carry[j];
  }
}

// Backward.  With G_t the gradient of h_t,
//   G_t = dh_t + a_{t+1} G_{t+1}   (G_{T-1} = dh_{T-1} + dh_last),
//   dx_t = G_t,  dlog_decay_t = a_t h_{t-1} G_t,  dh0 = a_0 G_0.
// What reaches token t from behind, R_t = a_{t+1} G_{t+1}, obeys the same kind
// of recurrence backwards in time with the same products A, so chunks are
// folded as in the forward kernel, last chunk first.  The saved output is
// rounded to its type, which would cost dlog_decay its precision; so h_{t-1}
// is formed again in fp32 from the state before the chunk, which the forward
// pass left in `ckpt` (4 bytes for every 64 tokens and channel).
template <typename TX, int V, bool CLUSTER>
__global__ void __launch_bounds__(kScanWarps * 32) scan_backward_kernel(ScanArgs a, int N) {
  __shared__ float2 part[2][kScanWarps][32 * V];  // each warp's (A, b) forwards
  __shared__ float back[2][kScanWarps][32 * V];   // and its b backwards
  __shared__ float2 tot[2][CLUSTER ? 16 : 1][32 * V];

  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
  const int c = (static_cast<int>(blockIdx.x) / N) * (32 * V) + lane * V;
  const int r = blockIdx.y;
  long long t0, n;
  if (!scan_row(a, r, blockIdx.x == 0 && threadIdx.x == 0, &t0, &n)) return;
  const bool live = c < a.C;

  float carry[V];  // R behind the cluster's current N chunks
#pragma unroll
  for (int j = 0; j < V; ++j)
    carry[j] = live && a.dh_last ? a.dh_last[static_cast<long long>(r) * a.C + c + j] : 0.f;

  const long long first = static_cast<long long>(rank) * kScanChunk + w * kScanTok;
  const long long stride = static_cast<long long>(N) * kScanChunk;
  const int steps = static_cast<int>((n + stride - 1) / stride);
  const TX* const dh = static_cast<const TX*>(a.dh);
  TX* const dx = static_cast<TX*>(a.dx);
  if constexpr (CLUSTER) cluster_sync();

  for (int s = steps - 1; s >= 0; --s) {
    const long long t = s * stride + first;
    const int buf = s & 1;
    ScanTile<TX, V> tile;
    Pack<TX, V> g[kScanTok];
    tile.load(a, t0, t, n, c, live);
    const long long at = (t0 + t) * a.C + c;
#pragma unroll
    for (int i = 0; i < kScanTok; ++i) {
      if (live && t + i < n) {
        g[i] = load_stream<TX, V>(dh + at + static_cast<long long>(i) * a.C);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) g[i].v[j] = from_f32<TX>(0.f);
      }
    }
    float base[V];  // state before this chunk
    {
      const long long chunk = t / kScanChunk;
#pragma unroll
      for (int j = 0; j < V; ++j)
        base[j] = live && chunk * kScanChunk < n ? a.ckpt[(t0 / kScanChunk + r + chunk) * a.C + c + j] : 0.f;
    }
    float al[kScanTok][V], A[V], b[V], e[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      A[j] = 1.f;
      b[j] = 0.f;
      e[j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kScanTok; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        al[i][j] = expf(tile.d[i].v[j]);
        b[j] = fmaf(al[i][j], b[j], to_f32(tile.x[i].v[j]));
        A[j] *= al[i][j];
      }
#pragma unroll
    for (int i = kScanTok - 1; i >= 0; --i)
#pragma unroll
      for (int j = 0; j < V; ++j) e[j] = al[i][j] * (to_f32(g[i].v[j]) + e[j]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      part[buf][w][lane * V + j] = make_float2(A[j], b[j]);
      back[buf][w][lane * V + j] = e[j];
    }
    __syncthreads();

    // state before this warp's tokens
    for (int i = 0; i < w; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float2 q = part[buf][i][lane * V + j];
        base[j] = fmaf(q.x, base[j], q.y);
      }
    // (pA, pe): the chunk's warps behind this one
    float pA[V], pe[V], R[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      pA[j] = 1.f;
      pe[j] = 0.f;
    }
    for (int i = kScanWarps - 1; i > w; --i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float q = part[buf][i][lane * V + j].x;
        pe[j] = fmaf(q, pe[j], back[buf][i][lane * V + j]);
        pA[j] *= q;
      }
    if constexpr (CLUSTER) {
      if (w == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float te = fmaf(A[j], pe[j], e[j]), tA = pA[j] * A[j];
          for (int q = 0; q < N; ++q) store_remote(remote_smem(&tot[buf][rank][lane * V + j], q), tA, te);
        }
      }
      cluster_sync();
#pragma unroll
      for (int j = 0; j < V; ++j) R[j] = carry[j];
      for (int q = N - 1; q >= 0; --q)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (q == rank) R[j] = carry[j];
          const float2 m = tot[buf][q][lane * V + j];
          carry[j] = fmaf(m.x, carry[j], m.y);
        }
    } else {
      float eA[V], ee[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        R[j] = carry[j];
        eA[j] = pA[j];
        ee[j] = pe[j];
      }
      for (int i = w; i >= 0; --i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float q = part[buf][i][lane * V + j].x;
          ee[j] = fmaf(q, ee[j], back[buf][i][lane * V + j]);
          eA[j] *= q;
        }
#pragma unroll
      for (int j = 0; j < V; ++j) carry[j] = fmaf(eA[j], carry[j], ee[j]);
    }

    float hp[kScanTok][V];  // a_t h_{t-1}
#pragma unroll
    for (int j = 0; j < V; ++j) R[j] = fmaf(pA[j], R[j], pe[j]);
#pragma unroll
    for (int i = 0; i < kScanTok; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        hp[i][j] = al[i][j] * base[j];
        base[j] = hp[i][j] + to_f32(tile.x[i].v[j]);
      }
#pragma unroll
    for (int i = kScanTok - 1; i >= 0; --i) {
      Pack<TX, V> ox;
      Pack<float, V> od;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float G = to_f32(g[i].v[j]) + R[j];
        ox.v[j] = from_f32<TX>(G);
        od.v[j] = hp[i][j] * G;
        R[j] = al[i][j] * G;
      }
      if (live && t + i < n) {
        store_stream<TX, V>(dx + at + static_cast<long long>(i) * a.C, ox);
        store_stream<float, V>(a.dlog_decay + at + static_cast<long long>(i) * a.C, od);
      }
    }
  }
  if (a.dh0 && live && rank == 0 && w == 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) a.dh0[static_cast<long long>(r) * a.C + c + j] = carry[j];
  }
}

// One token for every row: h = exp(log_decay) state + x, rounded to the
// output's type, and the fp32 state written back.  One thread for V channels;
// grid (channel tiles, rows).
template <typename TX, int V>
__global__ void __launch_bounds__(128) scan_step_kernel(ScanArgs a) {
  const int r = blockIdx.y;
  const int c = (static_cast<int>(blockIdx.x) * 128 + static_cast<int>(threadIdx.x)) * V;
  const int slot = row_slot(a.slot_idx, a.slots, r, a.err, blockIdx.x == 0 && threadIdx.x == 0);
  if (slot < 0 || c >= a.C) return;
  const long long in = static_cast<long long>(r) * a.C + c, st = static_cast<long long>(slot) * a.C + c;
  const auto x = load_stream<TX, V>(static_cast<const TX*>(a.x) + in);
  const auto d = load_stream<float, V>(a.log_decay + in);
  Pack<float, V> h = *reinterpret_cast<const Pack<float, V>*>(a.h0 + st);
  Pack<TX, V> o;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    h.v[j] = fmaf(expf(d.v[j]), h.v[j], to_f32(x.v[j]));
    o.v[j] = from_f32<TX>(h.v[j]);
  }
  *reinterpret_cast<Pack<float, V>*>(a.h_last + st) = h;
  *reinterpret_cast<Pack<TX, V>*>(static_cast<TX*>(a.h) + in) = o;
}

}  // namespace dl
