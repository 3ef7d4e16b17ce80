// Entry points of the paged-cache attention (kernels in paged.cuh).
#include "paged.cuh"
#include "launch.cuh"

#include <limits.h>
#include <math.h>

#include <initializer_list>

namespace {

using dl::PagedArgs;

int bad(const char* msg) { return dl::record_error(DL_ERR_ARG, msg); }
int unsupported(const char* msg) { return dl::record_error(DL_ERR_UNSUPPORTED, msg); }

int check(const int* slot_idx, int slots, int rows, int Hkv, int d, int dtype, int page_size, long long num_pages, int max_pages,
          const int* table) {
  if (dtype != DL_F32 && dtype != DL_BF16) return bad("unknown dtype");
  if (d != 64 && d != 128) return unsupported("d not in {64, 128}");
  if (rows < 0 || slots < 0 || Hkv < 1 || num_pages < 0 || max_pages < 0) return bad("negative size, or no key-value heads");
  if (rows > 65535) return unsupported("at most 65535 rows (grid y)");
  if (page_size < 1 || page_size > (1 << 20) || (page_size & (page_size - 1)))
    return unsupported("page_size not a power of two in [1, 2^20]");
  if (num_pages > 0 && static_cast<double>(num_pages) * Hkv * page_size >= 2147483648.0)
    return unsupported("2^31 or more rows of keys");
  if (num_pages > INT_MAX || Hkv > 65535) return unsupported("page ids are 32-bit, at most 65535 key-value heads");
  if (static_cast<long long>(max_pages) * page_size > (1 << 30)) return unsupported("more than 2^30 positions a slot");
  if (rows == 0) return DL_OK;
  if (slot_idx ? slots < 1 : slots < rows) return bad("fewer slots than rows");
  if (!table && max_pages > 0) return bad("null table");
  if (!dl::is_aligned(slot_idx, 4) || !dl::is_aligned(table, 4)) return bad("index pointer not 4-byte aligned");
  return DL_OK;
}

bool aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!dl::is_aligned(p, 16)) return false;
  return true;
}

int shift_of(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

constexpr int kSms = 148;

// How the tokens are shared out.
struct Split {
  int heads;        // query heads of a CTA
  int head_blocks;  // CTAs' head groups a key-value head
  bool even;        // equal runs of all tiles, through a workspace and a second launch
  int ctas;         // of the whole launch (even), else of a cluster
};

// Clusters of up to 8 CTAs, until the launch has three CTAs for every two SMs,
// as long as every warp finds two tiles in the longest row the table allows.
// The even form if a warp would then have more than eight.  B200, bf16, d = 128,
// 8 key-value heads of 4, clusters / even: 8 rows of 1024 tokens (4 tiles a
// warp) 13.5 / 16.8 us; 32 ragged rows of up to 4096 tokens (64) 65 / 54 us.
Split split_of(int rows, int G, int Hkv, int dtype, long long longest) {
  Split s{};
  s.heads = dtype == DL_BF16 ? (G > 8 ? 16 : 8) : G > 2 ? 4 : G;
  s.head_blocks = (G + s.heads - 1) / s.heads;
  const long long units = static_cast<long long>(rows) * Hkv * s.head_blocks;
  const long long tiles = (longest + dl::kTile - 1) / dl::kTile;
  s.ctas = 1;
  while (s.ctas < 8 && 2 * units * s.ctas < 3 * kSms && 2 * s.ctas * 4 * 2 <= tiles) s.ctas *= 2;
  if (tiles > 8 * 4 * s.ctas && rows <= dl::kPagedRows) {
    s.even = true;
    const long long runs = (units * (tiles + dl::kPagedStart) + dl::kPagedRun - 1) / dl::kPagedRun;  // most that have work
    const int resident = kSms * (s.heads > 8 ? 2 : 3);
    s.ctas = static_cast<int>(runs < resident ? runs : resident);
  }
  return s;
}

size_t plan_bytes(int rows) { return (sizeof(long long) * (rows + 2) + 15) / 16 * 16; }
size_t workspace_bytes(const Split& s, int rows, int d) {
  return s.even ? plan_bytes(rows) + sizeof(float) * 2 * s.ctas * s.heads * (d + 2) : 0;
}

long long longest_row(int max_pages, int page_size, int window) {
  const long long n = static_cast<long long>(max_pages) * page_size;
  return window > 0 && window < n ? window : n;
}

using Kernel = void (*)(PagedArgs, int);

template <typename T, int D, int HT>
cudaError_t launch(Kernel clusters, Kernel even, const PagedArgs& a, const Split& s, int warps, size_t smem, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(s.even ? even : clusters, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  if (!s.even)
    return dl::launch_cluster(clusters, dim3(static_cast<unsigned>(a.Hkv) * s.head_blocks * s.ctas, a.rows), warps * 32, smem, st, s.ctas,
                              a, s.ctas);
  even<<<s.ctas, warps * 32, smem, st>>>(a, 1);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 heads(a.Hkv * a.G, a.rows);
  // few units: each is cut into many pieces
  return static_cast<long long>(a.rows) * a.Hkv * s.head_blocks < kSms
             ? dl::launch_maybe_pdl(dl::paged_join_kernel<T, D, HT, 8>, heads, 8 * D, 0, st, true, a)
             : dl::launch_maybe_pdl(dl::paged_join_kernel<T, D, HT, 1>, heads, D, 0, st, true, a);
}

template <int D, int NT, int TT>
cudaError_t bf16(const PagedArgs& a, const Split& s, cudaStream_t st) {
  return launch<__nv_bfloat16, D, 8 * NT>(dl::paged_bf16_kernel<D, NT, 4, TT, false>, dl::paged_bf16_kernel<D, NT, 4, TT, true>, a, s, 4,
                                          sizeof(float) * 4 * 8 * NT * (D + 2), st);
}

template <int D, int HT>
cudaError_t f32(const PagedArgs& a, const Split& s, cudaStream_t st) {
  return launch<float, D, HT>(dl::paged_f32_kernel<D, HT, 4, false>, dl::paged_f32_kernel<D, HT, 4, true>, a, s, 4,
                              sizeof(float) * HT * (16 * (D + 2) + D), st);
}

// More than 4 heads a key are taken in blocks of 4, whose second reading comes
// from L2: 8 heads at once (8 dimensions a lane) took 64 rows of 8192 tokens from
// 772 to 687 us, but 4 rows of 4096 tokens from 43 to 67 us.
template <int D>
cudaError_t f32(const PagedArgs& a, const Split& s, cudaStream_t st) {
  return s.heads == 4 ? f32<D, 4>(a, s, st) : s.heads == 2 ? f32<D, 2>(a, s, st) : f32<D, 1>(a, s, st);
}

}  // namespace

extern "C" {

int dl_paged_attention(const int* slot_idx, int slots, int rows, int Hq, int Hkv, int d, int in_dtype, int page_size,
                       long long num_pages, int max_pages, const int* table, const int* lens, int window, float scale,
                       const void* q, const void* k, const void* v, void* k_pages, void* v_pages, void* out, void* workspace,
                       int* dev_err, void* stream) {
  const int rc = check(slot_idx, slots, rows, Hkv, d, in_dtype, page_size, num_pages, max_pages, table);
  if (rc != DL_OK) return rc;
  if (Hq < 1 || Hq % Hkv) return bad("Hq not a positive multiple of Hkv");
  if (window < 0) return bad("negative window");
  if (!(fabsf(scale) <= 3.0e38f)) return bad("scale is not finite");
  if (rows == 0) return DL_OK;
  if (!lens || !q || !out || (num_pages > 0 && (!k_pages || !v_pages))) return bad("null input/output pointer");
  if ((k == nullptr) != (v == nullptr)) return bad("k and v go together");
  if (!aligned16({q, k, v, k_pages, v_pages, out})) return bad("pointer not 16-byte aligned");
  if (!dl::is_aligned(lens, 4) || !dl::is_aligned(dev_err, 4)) return bad("int pointer not 4-byte aligned");
  if (!dl::is_aligned(workspace, 16)) return bad("workspace not 16-byte aligned");
  Split s = split_of(rows, Hq / Hkv, Hkv, in_dtype, longest_row(max_pages, page_size, window));
  if (s.even && !workspace) {  // the widest form without one
    s.even = false;
    s.ctas = 8;
  }
  PagedArgs a{};
  a.q = q;
  a.k_new = k;
  a.v_new = v;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.table = table;
  a.lens = lens;
  a.slot_idx = slot_idx;
  a.out = out;
  a.err = dev_err;
  a.pages = num_pages;
  a.slots = slots;
  a.max_pages = max_pages;
  a.page_shift = shift_of(page_size);
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.window = window;
  a.scale = scale * 1.44269504088896340736f;  // exponents in base 2
  a.head_blocks = s.head_blocks;
  a.rows = rows;
  if (s.even) {
    a.plan = static_cast<long long*>(workspace);
    a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan_bytes(rows));
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (in_dtype == DL_BF16) {
    if (d == 128) e = s.heads == 8 ? bf16<128, 1, 1>(a, s, st) : bf16<128, 2, 1>(a, s, st);
    else e = s.heads == 8 ? bf16<64, 1, 2>(a, s, st) : bf16<64, 2, 2>(a, s, st);
  } else {
    e = d == 128 ? f32<128>(a, s, st) : f32<64>(a, s, st);
  }
  return e == cudaSuccess ? DL_OK : dl::launch_failed(e, "paged attention launch");
}

int dl_paged_attention_workspace(int rows, int Hq, int Hkv, int d, int in_dtype, int page_size, int max_pages, int window,
                                 size_t* bytes) {
  if (!bytes) return bad("null output pointer");
  if (rows < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv || d < 1 || page_size < 1 || max_pages < 0 || window < 0 ||
      (in_dtype != DL_F32 && in_dtype != DL_BF16))
    return bad("bad size or dtype");
  *bytes = rows ? workspace_bytes(split_of(rows, Hq / Hkv, Hkv, in_dtype, longest_row(max_pages, page_size, window)), rows, d) : 0;
  return DL_OK;
}

int dl_paged_write(const int* slot_idx, int slots, int rows, const int* cu_seqlens, long long total, int Hkv, int d,
                   int in_dtype, int page_size, long long num_pages, int max_pages, const int* table, const int* starts,
                   const void* k, const void* v, void* k_pages, void* v_pages, int* dev_err, void* stream) {
  const int rc = check(slot_idx, slots, rows, Hkv, d, in_dtype, page_size, num_pages, max_pages, table);
  if (rc != DL_OK) return rc;
  if (total < 0 || total > INT_MAX) return bad("total outside [0, 2^31)");
  if (rows == 0 || total == 0) return DL_OK;
  if (!cu_seqlens || !k || !v || !k_pages || !v_pages) return bad("null input/output pointer");
  if (!aligned16({k, v, k_pages, v_pages})) return bad("pointer not 16-byte aligned");
  if (!dl::is_aligned(cu_seqlens, 4) || !dl::is_aligned(starts, 4) || !dl::is_aligned(dev_err, 4))
    return bad("int pointer not 4-byte aligned");
  PagedArgs a{};
  a.k = k;
  a.v = v;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.table = table;
  a.slot_idx = slot_idx;
  a.cu = cu_seqlens;
  a.starts = starts;
  a.err = dev_err;
  a.total = total;
  a.pages = num_pages;
  a.slots = slots;
  a.max_pages = max_pages;
  a.page_shift = shift_of(page_size);
  a.Hkv = Hkv;
  const int row_units = d * (in_dtype == DL_BF16 ? 2 : 4) / 16;
  const long long ctas = (total * Hkv * row_units / rows + 256 * 8 - 1) / (256 * 8);  // eight 16-byte units a thread
  const int x = static_cast<int>(ctas < 1 ? 1 : ctas > 148 * 8 ? 148 * 8 : ctas);
  dl::paged_write_kernel<<<dim3(x, rows), 256, 0, static_cast<cudaStream_t>(stream)>>>(a, row_units);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DL_OK : dl::launch_failed(e, "paged write launch");
}

}  // extern "C"
