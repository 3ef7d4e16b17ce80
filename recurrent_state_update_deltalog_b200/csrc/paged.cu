// Entry points of the paged-cache attention (kernels in paged.cuh).
#include "paged.cuh"

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
  if (num_pages > INT_MAX || Hkv > 65535) return unsupported("page ids are 32-bit, at most 65535 key-value heads");
  if (static_cast<long long>(max_pages) * page_size > INT_MAX - 65536) return unsupported("positions are 32-bit");
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

// Launches one kernel with N CTAs a cluster.
cudaError_t launch(void (*kern)(PagedArgs, int), const PagedArgs& a, int rows, int warps, size_t smem, int N, cudaStream_t st) {
  if (smem + 1024 > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return dl::launch_cluster(kern, dim3(static_cast<unsigned>(a.Hkv) * a.head_blocks * N, rows), warps * 32, smem, st, N, a, N);
}

template <int D, int NT, int W, int TT>
cudaError_t bf16(const PagedArgs& a, int rows, int N, cudaStream_t st) {
  return launch(dl::paged_bf16_kernel<D, NT, W, TT>, a, rows, W, sizeof(float) * W * 8 * NT * (D + 2), N, st);
}

template <int D, int HT, int W>
cudaError_t f32(const PagedArgs& a, int rows, int N, cudaStream_t st) {
  return launch(dl::paged_f32_kernel<D, HT, W>, a, rows, W, sizeof(float) * HT * (W * 4 * (D + 2) + D), N, st);
}

// CTAs a (row, head group): enough for about three CTAs an SM, no more than
// the longest possible row has work for (`most` warps' shares).
int cluster_of(long long units, int warps, long long most) {
  int n = 1;
  while (n < 8 && units * n < 3 * 148 && 2ll * n * warps <= most) n *= 2;
  return n;
}

}  // namespace

extern "C" {

int dl_paged_attention(const int* slot_idx, int slots, int rows, int Hq, int Hkv, int d, int in_dtype, int page_size,
                       long long num_pages, int max_pages, const int* table, const int* lens, int window, float scale,
                       const void* q, const void* k, const void* v, void* k_pages, void* v_pages, void* out, int* dev_err,
                       void* stream) {
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
  long long longest = static_cast<long long>(max_pages) * page_size;
  if (window > 0 && window < longest) longest = window;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (in_dtype == DL_BF16) {
    const int nt = a.G > 8 ? 2 : 1;
    a.head_blocks = (a.G + 8 * nt - 1) / (8 * nt);
    const int n = cluster_of(static_cast<long long>(rows) * Hkv * a.head_blocks, 4, longest / 32);
    if (d == 128) e = nt == 1 ? bf16<128, 1, 4, 1>(a, rows, n, st) : bf16<128, 2, 4, 1>(a, rows, n, st);
    else e = nt == 1 ? bf16<64, 1, 4, 2>(a, rows, n, st) : bf16<64, 2, 4, 2>(a, rows, n, st);
  } else {
    const int ht = a.G > 2 ? 4 : a.G;
    a.head_blocks = (a.G + ht - 1) / ht;
    const int n = cluster_of(static_cast<long long>(rows) * Hkv * a.head_blocks, 16, longest / 4);
    if (d == 128)
      e = ht == 4 ? f32<128, 4, 4>(a, rows, n, st) : ht == 2 ? f32<128, 2, 4>(a, rows, n, st) : f32<128, 1, 4>(a, rows, n, st);
    else
      e = ht == 4 ? f32<64, 4, 4>(a, rows, n, st) : ht == 2 ? f32<64, 2, 4>(a, rows, n, st) : f32<64, 1, 4>(a, rows, n, st);
  }
  return e == cudaSuccess ? DL_OK : dl::launch_failed(e, "paged attention launch");
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
