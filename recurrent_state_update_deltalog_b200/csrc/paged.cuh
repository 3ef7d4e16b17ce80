// Attention of one new token a sequence over a paged key-value cache, with the
// write of that token's key and value, split over the cache's length and
// joined in one launch; and the copy of prompts into the pages.
//
// For query head h of key-value head g, over the tokens j that the length and
// the window leave, o_h = sum_j p_j v_j / sum_j p_j, p_j = exp(s_j - m),
// s_j = scale q_h . k_j, m = max s_j.  Each warp keeps a running (m, sum p,
// sum p v) over its tokens; two such triples join by scaling both to the
// larger m, so any split of the tokens gives the same value up to rounding.
//
// Bound: memory; each key and value is read once for all query heads of its
// group (4 G flops an element of 2 bytes).  The tokens of one (row, key-value
// head) are dealt out in tiles of 16 to the warps of a cluster of CTAs, whose
// triples meet in distributed shared memory: one launch, no workspace, no
// atomics, results independent of timing.
//
// bf16: warp MMAs (m16n8k16) with the cache as the 16-row operand and 8 query
// heads as the columns, S^T = K Q^T and O^T = V^T P^T.  The contraction over
// the head dimension may run in any order, so a lane's 16-byte load of a key
// is its fragment of two MMAs as it stands; the rows of O^T may stand in any
// order, so 16-byte loads of four values need only byte permutes within the
// lane.  P^T is S^T transposed in registers (movmatrix).  Nothing passes
// through shared memory before the join.  tcgen05 would want 64 or 128 rows of
// queries and staged operands; at 8 heads the tensor work is far below the
// loads either way.  fp32: FMAs, 8 lanes a key.
#pragma once

#include "ops.cuh"

namespace dl {

struct PagedArgs {
  const void* q;          // [rows][Hq][d]
  const void* k_new;      // [rows][Hkv][d] or null
  const void* v_new;
  void* k_pages;          // [pages][Hkv][page][d]
  void* v_pages;
  const int* table;       // [slots][max_pages]
  const int* lens;        // [slots] tokens, the new one included
  const int* slot_idx;    // [rows] or null
  void* out;              // [rows][Hq][d]
  int* err;
  long long pages;
  int slots, max_pages, page_shift;
  int Hkv, G;             // G = Hq / Hkv query heads a key-value head
  int head_blocks;        // CTAs' head groups a key-value head
  int window;             // 0: none
  float scale;            // times log2(e)
  // prompts
  const int* cu;          // [rows + 1]
  const int* starts;      // [slots] position of each row's first token
  const void* k;          // [total][Hkv][d]
  const void* v;
  long long total;
};

__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(gmem_u64(p)));
  return r;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  uint32_t u;
  memcpy(&u, &p, 4);
  return u;
}

__device__ __forceinline__ float load_remote(uint32_t addr) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
  return x;
}

// 2^x, and 0 for -inf; the first operand may be -inf like the second.
__device__ __forceinline__ float exp2_diff(float x, float m) { return m == -INFINITY ? 0.f : exp2f(x - m); }

// Page of position `pos` of a slot's table row, or -1 (reported).
__device__ __forceinline__ long long page_of(const PagedArgs& a, const int* table, int pos) {
  const int p = __ldg(table + (pos >> a.page_shift));
  if (p < 0 || p >= a.pages) {
    raise_error(a.err, DL_DEVERR_PAGE);
    return -1;
  }
  return p;
}

// A row's slot and its tokens [first, len); false: the row is skipped.
__device__ __forceinline__ bool paged_row(const PagedArgs& a, int r, bool tell, int* slot, int* first, int* len) {
  *slot = row_slot(a.slot_idx, a.slots, r, a.err, tell);
  if (*slot < 0) return false;
  const int n = __ldg(a.lens + *slot);
  if (n < 0 || n > (static_cast<long long>(a.max_pages) << a.page_shift)) {
    if (tell) raise_error(a.err, DL_DEVERR_SEQLEN);
    return false;
  }
  *len = n;
  *first = a.window > 0 && n > a.window ? n - a.window : 0;
  return true;
}

// Stores the new token's key and value of one (row, key-value head).
template <typename T, int D>
__device__ __forceinline__ void store_new(const PagedArgs& a, int r, int kvh, const int* table, int len) {
  constexpr int U = D * sizeof(T) / 16;  // 16-byte units
  if (threadIdx.x >= 2 * U || len < 1) return;
  const long long page = page_of(a, table, len - 1);
  if (page < 0) return;
  const int u = threadIdx.x % U;
  const bool val = threadIdx.x >= U;
  const long long at = (((page * a.Hkv + kvh) << a.page_shift) + ((len - 1) & ((1 << a.page_shift) - 1))) * D;
  T* const to = static_cast<T*>(val ? a.v_pages : a.k_pages) + at;
  const T* const from = static_cast<const T*>(val ? a.v_new : a.k_new) + (static_cast<long long>(r) * a.Hkv + kvh) * D;
  reinterpret_cast<uint4*>(to)[u] = reinterpret_cast<const uint4*>(from)[u];
}

// Joins the NP triples of this CTA and then those of the cluster's N CTAs, and
// writes the outputs of heads [h0, h0 + HT).  `o` [NP][HT][D], `ml` [NP][HT][2].
template <typename T, int D, int HT, int NP, int THREADS>
__device__ __forceinline__ void join_and_store(const PagedArgs& a, float* o, float* ml, int r, int kvh, int h0, int N, int rank) {
  __syncthreads();
  __shared__ float top[HT][2];  // the CTA's (m, sum)
  for (int h = threadIdx.x; h < HT; h += THREADS) {
    float m = -INFINITY, l = 0.f;
    for (int p = 0; p < NP; ++p) m = fmaxf(m, ml[(p * HT + h) * 2]);
    for (int p = 0; p < NP; ++p) l += ml[(p * HT + h) * 2 + 1] * exp2_diff(ml[(p * HT + h) * 2], m);
    top[h][0] = m;
    top[h][1] = l;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < HT * D; e += THREADS) {
    const int h = e / D;
    float s = 0.f;
#pragma unroll 4
    for (int p = 0; p < NP; ++p) s += o[p * HT * D + e] * exp2_diff(ml[(p * HT + h) * 2], top[h][0]);
    o[e] = s;  // element e of the first triple is read by this thread alone
  }
  if (N > 1) cluster_sync();
  else __syncthreads();
  const int share = HT * D / N;  // N divides 8, HT * D is a multiple of 64
  for (int i = threadIdx.x; i < share; i += THREADS) {
    const int e = rank * share + i, h = e / D;
    if (h0 + h >= a.G) continue;
    float m = -INFINITY, l = 0.f, s = 0.f;
    for (int q = 0; q < N; ++q) m = fmaxf(m, N > 1 ? load_remote(remote_smem(&top[h][0], q)) : top[h][0]);
    for (int q = 0; q < N; ++q) {
      const float w = exp2_diff(N > 1 ? load_remote(remote_smem(&top[h][0], q)) : top[h][0], m);
      l += w * (N > 1 ? load_remote(remote_smem(&top[h][1], q)) : top[h][1]);
      s += w * (N > 1 ? load_remote(remote_smem(o + e, q)) : o[e]);
    }
    const long long head = static_cast<long long>(r) * a.Hkv * a.G + static_cast<long long>(kvh) * a.G + h0 + h;
    static_cast<T*>(a.out)[head * D + e % D] = from_f32<T>(l == 0.f ? 0.f : s / l);
  }
  if (N > 1) cluster_sync();  // no CTA leaves while another reads its shared memory
}

// bf16.  Grid (Hkv * head_blocks * N, rows), clusters of N; W warps a CTA; NT
// column tiles of 8 query heads; tiles of 16 tokens, TT at a time.
template <int D, int NT, int W, int TT>
__global__ void __launch_bounds__(W * 32) paged_bf16_kernel(PagedArgs a, int N) {
  constexpr int HT = 8 * NT, KB = D / 32, VB = D / 64;
  using bf16 = __nv_bfloat16;
  extern __shared__ float smem[];  // o [W][HT][D], ml [W][HT][2]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, j = lane % 4;
  const int rank = N > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int unit = static_cast<int>(blockIdx.x) / N, kvh = unit / a.head_blocks, h0 = (unit % a.head_blocks) * HT;
  const int r = blockIdx.y;
  int slot, first, len;
  if (!paged_row(a, r, blockIdx.x == 0 && threadIdx.x == 0, &slot, &first, &len)) return;  // the whole cluster
  const int* const table = a.table + static_cast<long long>(slot) * a.max_pages;
  if (a.k_new && rank == 0 && unit % a.head_blocks == 0) store_new<bf16, D>(a, r, kvh, table, len);

  uint32_t q[NT][KB][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const int h = h0 + t * 8 + g;
      uint4 u = make_uint4(0, 0, 0, 0);
      if (h < a.G) u = ld16(static_cast<const bf16*>(a.q) + (static_cast<long long>(r) * a.Hkv * a.G + kvh * a.G + h) * D + b * 32 + j * 8);
      q[t][b][0] = u.x;
      q[t][b][1] = u.y;
      q[t][b][2] = u.z;
      q[t][b][3] = u.w;
    }
  float o[NT][VB][4][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t][0] = m[t][1] = -INFINITY;
    l[t][0] = l[t][1] = 0.f;
#pragma unroll
    for (int b = 0; b < VB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[t][b][i][c] = 0.f;
  }

  const long long new_at = (static_cast<long long>(r) * a.Hkv + kvh) * D;
  const int mask = (1 << a.page_shift) - 1;
  // Rows of keys and values of position `pos` (null: not there).
  auto rows_of = [&](int pos, const bf16** kr, const bf16** vr) {
    *kr = *vr = nullptr;
    if (pos < first || pos >= len) return;
    if (a.k_new && pos == len - 1) {
      *kr = static_cast<const bf16*>(a.k_new) + new_at;
      *vr = static_cast<const bf16*>(a.v_new) + new_at;
      return;
    }
    const long long page = page_of(a, table, pos);
    if (page < 0) return;
    const long long at = (((page * a.Hkv + kvh) << a.page_shift) + (pos & mask)) * D;
    *kr = static_cast<const bf16*>(a.k_pages) + at;
    *vr = static_cast<const bf16*>(a.v_pages) + at;
  };

  const int tile0 = first / 16, tiles = len > 0 ? (len + 15) / 16 : 0;
  for (int tile = tile0 + (rank * W + warp) * TT; tile < tiles; tile += N * W * TT) {
    uint4 kf[TT][2][KB], vf[TT][4][VB];
    bool there[TT][2];  // of this lane's two score rows
#pragma unroll
    for (int x = 0; x < TT; ++x) {
      const int pos = (tile + x) * 16;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bf16 *kr, *vr;
        rows_of(pos + g + s * 8, &kr, &vr);
        there[x][s] = kr != nullptr;
#pragma unroll
        for (int b = 0; b < KB; ++b) kf[x][s][b] = kr ? ld16(kr + b * 32 + j * 8) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bf16 *kr, *vr;
        rows_of(pos + 2 * j + (s & 1) + (s >> 1) * 8, &kr, &vr);
#pragma unroll
        for (int b = 0; b < VB; ++b) vf[x][s][b] = vr ? ld16(vr + b * 64 + g * 8) : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float s[TT][4];
#pragma unroll
      for (int x = 0; x < TT; ++x) {
        s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.f;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
          mma16816(s[x], kf[x][0][b].x, kf[x][1][b].x, kf[x][0][b].y, kf[x][1][b].y, q[t][b][0], q[t][b][1]);
          mma16816(s[x], kf[x][0][b].z, kf[x][1][b].z, kf[x][0][b].w, kf[x][1][b].w, q[t][b][2], q[t][b][3]);
        }
      }
      float top[2] = {m[t][0], m[t][1]};
#pragma unroll
      for (int x = 0; x < TT; ++x)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s[x][c] = there[x][c >> 1] ? s[x][c] * a.scale : -INFINITY;
          top[c & 1] = fmaxf(top[c & 1], s[x][c]);
        }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[c] = fmaxf(top[c], __shfl_xor_sync(~0u, top[c], 4));
        top[c] = fmaxf(top[c], __shfl_xor_sync(~0u, top[c], 8));
        top[c] = fmaxf(top[c], __shfl_xor_sync(~0u, top[c], 16));
        const float w = exp2_diff(m[t][c], top[c]);
        m[t][c] = top[c];
        l[t][c] *= w;
#pragma unroll
        for (int b = 0; b < VB; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[t][b][i][c] *= w;
            o[t][b][i][c + 2] *= w;
          }
      }
#pragma unroll
      for (int x = 0; x < TT; ++x) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s[x][c] = exp2_diff(s[x][c], m[t][c & 1]);
          l[t][c & 1] += s[x][c];
        }
        const uint32_t b0 = transpose8x8(pack_bf16(s[x][0], s[x][1])), b1 = transpose8x8(pack_bf16(s[x][2], s[x][3]));
#pragma unroll
        for (int b = 0; b < VB; ++b) {
          const uint32_t* const v0 = reinterpret_cast<const uint32_t*>(&vf[x][0][b]);
          const uint32_t* const v1 = reinterpret_cast<const uint32_t*>(&vf[x][1][b]);
          const uint32_t* const v2 = reinterpret_cast<const uint32_t*>(&vf[x][2][b]);
          const uint32_t* const v3 = reinterpret_cast<const uint32_t*>(&vf[x][3][b]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma16816(o[t][b][i], __byte_perm(v0[i], v1[i], 0x5410), __byte_perm(v0[i], v1[i], 0x7632),
                     __byte_perm(v2[i], v3[i], 0x5410), __byte_perm(v2[i], v3[i], 0x7632), b0, b1);
        }
      }
    }
  }

  float* const so = smem + warp * HT * D;
  float* const ml = smem + W * HT * D;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float sum = l[t][c];
      sum += __shfl_xor_sync(~0u, sum, 4);
      sum += __shfl_xor_sync(~0u, sum, 8);
      sum += __shfl_xor_sync(~0u, sum, 16);
      const int h = t * 8 + 2 * j + c;
      if (g == 0) {
        ml[(warp * HT + h) * 2] = m[t][c];
        ml[(warp * HT + h) * 2 + 1] = sum;
      }
#pragma unroll
      for (int b = 0; b < VB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          so[h * D + b * 64 + g * 8 + 2 * i] = o[t][b][i][c];
          so[h * D + b * 64 + g * 8 + 2 * i + 1] = o[t][b][i][c + 2];
        }
    }
  join_and_store<bf16, D, HT, W, W * 32>(a, smem, ml, r, kvh, h0, N, rank);
}

// fp32.  8 lanes a token, D / 8 dimensions each (4 of every 32); every group
// of 8 lanes keeps its own triple for HT query heads.
template <int D, int HT, int W>
__global__ void __launch_bounds__(W * 32) paged_f32_kernel(PagedArgs a, int N) {
  constexpr int B = D / 32, NP = W * 4;
  extern __shared__ float smem[];  // o [NP][HT][D], ml [NP][HT][2], q [HT][D]
  const int grp = threadIdx.x / 8, lane = threadIdx.x % 8;
  const int rank = N > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int unit = static_cast<int>(blockIdx.x) / N, kvh = unit / a.head_blocks, h0 = (unit % a.head_blocks) * HT;
  const int r = blockIdx.y;
  int slot, first, len;
  if (!paged_row(a, r, blockIdx.x == 0 && threadIdx.x == 0, &slot, &first, &len)) return;
  const int* const table = a.table + static_cast<long long>(slot) * a.max_pages;
  if (a.k_new && rank == 0 && unit % a.head_blocks == 0) store_new<float, D>(a, r, kvh, table, len);

  float* const ml = smem + NP * HT * D;
  float* const sq = ml + NP * HT * 2;
  for (int e = threadIdx.x; e < HT * D; e += W * 32)
    sq[e] = h0 + e / D < a.G
                ? static_cast<const float*>(a.q)[(static_cast<long long>(r) * a.Hkv * a.G + kvh * a.G + h0) * D + e] * a.scale
                : 0.f;
  __syncthreads();
  float o[HT][B][4], m[HT], l[HT];
#pragma unroll
  for (int h = 0; h < HT; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[h][b][i] = 0.f;
  }
  const long long new_at = (static_cast<long long>(r) * a.Hkv + kvh) * D;
  const int mask = (1 << a.page_shift) - 1, step = N * NP;
  // the loop's length is the warp's, not the group's: its shuffles take every lane
  for (int base = first + (rank * NP + grp / 4 * 4); base < len; base += step) {
    const int pos = base + grp % 4;
    const float *kr = nullptr, *vr = nullptr;
    if (pos < len) {
      if (a.k_new && pos == len - 1) {
        kr = static_cast<const float*>(a.k_new) + new_at;
        vr = static_cast<const float*>(a.v_new) + new_at;
      } else {
        const long long page = page_of(a, table, pos);
        if (page >= 0) {
          const long long at = (((page * a.Hkv + kvh) << a.page_shift) + (pos & mask)) * D;
          kr = static_cast<const float*>(a.k_pages) + at;
          vr = static_cast<const float*>(a.v_pages) + at;
        }
      }
    }
    float kf[B][4], vf[B][4];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const uint4 uk = kr ? ld16(kr + b * 32 + lane * 4) : make_uint4(0, 0, 0, 0);
      const uint4 uv = vr ? ld16(vr + b * 32 + lane * 4) : make_uint4(0, 0, 0, 0);
      memcpy(kf[b], &uk, 16);
      memcpy(vf[b], &uv, 16);
    }
#pragma unroll
    for (int h = 0; h < HT; ++h) {
      float s = 0.f;
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const float4 x = *reinterpret_cast<const float4*>(sq + h * D + b * 32 + lane * 4);
        s = fmaf(kf[b][0], x.x, s);
        s = fmaf(kf[b][1], x.y, s);
        s = fmaf(kf[b][2], x.z, s);
        s = fmaf(kf[b][3], x.w, s);
      }
      s += __shfl_xor_sync(~0u, s, 1);
      s += __shfl_xor_sync(~0u, s, 2);
      s += __shfl_xor_sync(~0u, s, 4);
      if (!kr) s = -INFINITY;
      const float top = fmaxf(m[h], s), w = exp2_diff(m[h], top), p = exp2_diff(s, top);
      m[h] = top;
      l[h] = fmaf(l[h], w, p);
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[h][b][i] = fmaf(p, vf[b][i], o[h][b][i] * w);
    }
  }
#pragma unroll
  for (int h = 0; h < HT; ++h) {
    if (lane == 0) {
      ml[(grp * HT + h) * 2] = m[h];
      ml[(grp * HT + h) * 2 + 1] = l[h];
    }
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) smem[(grp * HT + h) * D + b * 32 + lane * 4 + i] = o[h][b][i];
  }
  join_and_store<float, D, HT, NP, W * 32>(a, smem, ml, r, kvh, h0, N, rank);
}

// Prompts into the pages: row r's tokens [cu[r], cu[r + 1]) go to positions
// starts[slot] + 0, 1, ...; grid (CTAs a row, rows), 16 bytes a thread.
__global__ void __launch_bounds__(256) paged_write_kernel(PagedArgs a, int row_units) {
  const int r = blockIdx.y;
  const bool tell = blockIdx.x == 0 && threadIdx.x == 0;
  const int slot = row_slot(a.slot_idx, a.slots, r, a.err, tell);
  if (slot < 0) return;
  const int s = __ldg(a.cu + r), e = __ldg(a.cu + r + 1), start = a.starts ? __ldg(a.starts + slot) : 0;
  if (s < 0 || e < s || e > a.total || start < 0 ||
      static_cast<long long>(start) + e - s > (static_cast<long long>(a.max_pages) << a.page_shift)) {
    if (tell) raise_error(a.err, DL_DEVERR_SEQLEN);
    return;
  }
  const int* const table = a.table + static_cast<long long>(slot) * a.max_pages;
  const int mask = (1 << a.page_shift) - 1;
  const long long units = static_cast<long long>(e - s) * a.Hkv * row_units;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < units; i += static_cast<long long>(gridDim.x) * 256) {
    const int u = static_cast<int>(i % row_units);
    const long long th = i / row_units;
    const int h = static_cast<int>(th % a.Hkv), pos = start + static_cast<int>(th / a.Hkv);
    const long long page = page_of(a, table, pos);
    if (page < 0) continue;
    const long long from = static_cast<long long>(s) * a.Hkv * row_units + i;
    const long long to = (((page * a.Hkv + h) << a.page_shift) + (pos & mask)) * row_units + u;
    static_cast<uint4*>(a.k_pages)[to] = ld16(static_cast<const uint4*>(a.k) + from);
    static_cast<uint4*>(a.v_pages)[to] = ld16(static_cast<const uint4*>(a.v) + from);
  }
}

}  // namespace dl
