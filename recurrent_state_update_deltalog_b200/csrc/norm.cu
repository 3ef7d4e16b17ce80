// Entry points of the norms around a block (kernels in norm.cuh).
#include "norm.cuh"

#include <initializer_list>

namespace {

using dl::NormArgs;

int bad(const char* msg) { return dl::record_error(DL_ERR_ARG, msg); }

// How a row of n channels lies on threads: V channels a load, nv loads a
// thread, tpr threads a row.
struct Shape {
  int vec, nv, tpr;
  bool narrow;
  int block() const { return narrow ? dl::kNormNarrow : tpr; }
  int rows_per_cta() const { return narrow ? dl::kNormNarrow / tpr : 1; }
};

Shape shape_of(int n, int dtype, bool wide_loads) {
  Shape s{};
  s.vec = wide_loads ? (dtype == DL_BF16 ? 8 : 4) : 1;
  const int loads = (n + s.vec - 1) / s.vec;
  s.nv = 1;
  while (s.nv < 8 && loads > 512 * s.nv) s.nv *= 2;
  s.narrow = loads <= 32;
  if (s.narrow) {
    s.tpr = 8;
    while (s.tpr < loads) s.tpr *= 2;
  } else {
    s.tpr = ((loads + s.nv - 1) / s.nv + 31) / 32 * 32;
  }
  return s;
}

bool wide_loads(int n, int dtype, std::initializer_list<const void*> tensors, std::initializer_list<const void*> weights) {
  if (n % (dtype == DL_BF16 ? 8 : 4)) return false;
  for (const void* p : tensors)
    if (!dl::is_aligned(p, 16)) return false;
  for (const void* p : weights)
    if (!dl::is_aligned(p, 16)) return false;
  return true;
}

// CTAs of the backward kernel: a few an SM, no more than there are rows.  The
// bound is the same for every alignment, so that the workspace is too.
int backward_ctas(long long rows, const Shape& s) {
  const int per_sm = s.narrow ? 4 : (s.tpr > 512 ? 1 : 1024 / s.tpr > 8 ? 8 : 1024 / s.tpr);
  const long long need = (rows + s.rows_per_cta() - 1) / s.rows_per_cta();
  const long long most = 148ll * per_sm;
  return static_cast<int>(need < most ? need : most);
}
constexpr int kMostCtas = 148 * 8;

int check(int rows, int D, int groups, int dtype, const void* y, const float* scale, const float* pre, float eps) {
  if (dtype != DL_F32 && dtype != DL_BF16) return bad("unknown dtype");
  if (rows < 0 || D < 1 || groups < 1 || D % groups) return bad("rows < 0, D < 1, or D not a multiple of groups");
  if (D / groups > dl::kNormMax) return dl::record_error(DL_ERR_UNSUPPORTED, "more than 8192 channels a group");
  if (groups > 1 && (scale || pre))
    return dl::record_error(DL_ERR_UNSUPPORTED, "scale and pre weights need groups = 1");
  if (!(eps >= 0.f)) return bad("eps is negative or not a number");
  if (rows > 0 && !y) return bad("null y");
  if (static_cast<long long>(rows) * groups > 0x7fffffffll) return dl::record_error(DL_ERR_UNSUPPORTED, "rows * groups past 2^31 - 1");
  return DL_OK;
}

bool ok_typed(int dtype, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!dl::is_aligned(p, dtype == DL_BF16 ? 2 : 4)) return false;
  return true;
}

template <typename T, int V, int NV, bool NARROW>
cudaError_t run(const NormArgs& a, const Shape& s, int ctas, bool back, cudaStream_t st) {
  if (back) {
    const size_t smem = NARROW && a.partial ? static_cast<size_t>(s.rows_per_cta()) * a.n * 4 : 0;
    dl::norm_backward_kernel<T, V, NV, NARROW><<<ctas, s.block(), smem, st>>>(a);
  } else {
    dl::norm_kernel<T, V, NV, NARROW><<<ctas, s.block(), 0, st>>>(a);
  }
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t run(const NormArgs& a, const Shape& s, int ctas, bool back, cudaStream_t st) {
  if (s.narrow) return run<T, V, 1, true>(a, s, ctas, back, st);
  switch (s.nv) {
    case 1: return run<T, V, 1, false>(a, s, ctas, back, st);
    case 2: return run<T, V, 2, false>(a, s, ctas, back, st);
    case 4:
      if constexpr (V < 8) return run<T, V, 4, false>(a, s, ctas, back, st);
      break;
    default:
      if constexpr (V < 4) return run<T, V, 8, false>(a, s, ctas, back, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t run(const NormArgs& a, const Shape& s, int ctas, int dtype, bool back, cudaStream_t st) {
  if (dtype == DL_BF16)
    return s.vec > 1 ? run<__nv_bfloat16, 8>(a, s, ctas, back, st) : run<__nv_bfloat16, 1>(a, s, ctas, back, st);
  return s.vec > 1 ? run<float, 4>(a, s, ctas, back, st) : run<float, 1>(a, s, ctas, back, st);
}

}  // namespace

extern "C" {

int dl_block_norm(const int* slot_idx, int slots, int rows, int D, int groups, int in_dtype, const void* y,
                  const float* post_weight, const void* gate, const float* scale, const void* residual,
                  const float* pre_weight, float eps, void* out, void* normed, void* stream) {
  const int rc = check(rows, D, groups, in_dtype, y, scale, pre_weight, eps);
  if (rc != DL_OK) return rc;
  if (rows == 0) return DL_OK;
  if (slot_idx && slots < 1) return bad("slot map without slots");
  if (!out && !pre_weight) return bad("null out");
  if ((pre_weight != nullptr) != (normed != nullptr)) return bad("normed goes with a pre weight");
  if (!ok_typed(in_dtype, {y, gate, residual, out, normed}) ||
      !ok_typed(DL_F32, {post_weight, scale, pre_weight, slot_idx}))
    return bad("pointer not aligned to its element size");
  NormArgs a{};
  a.y = y;
  a.gate = gate;
  a.residual = residual;
  a.post = post_weight;
  a.scale = scale;
  a.pre = pre_weight;
  a.out = out;
  a.normed = normed;
  a.slot_idx = slot_idx;
  a.slots = slots;
  a.groups = groups;
  a.n = D / groups;
  a.rows = static_cast<long long>(rows) * groups;
  a.eps = eps;
  const Shape s = shape_of(a.n, in_dtype, wide_loads(a.n, in_dtype, {y, gate, residual, out, normed}, {post_weight, scale, pre_weight}));
  a.tpr = s.tpr;
  const int ctas = static_cast<int>((a.rows + s.rows_per_cta() - 1) / s.rows_per_cta());
  const cudaError_t e = run(a, s, ctas, in_dtype, false, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DL_OK : dl::launch_failed(e, "block norm launch");
}

int dl_block_norm_workspace(int rows, int D, int groups, size_t* bytes) {
  if (!bytes) return bad("null output pointer");
  if (rows < 0 || D < 1 || groups < 1 || D % groups) return bad("rows < 0, D < 1, or D not a multiple of groups");
  const long long units = static_cast<long long>(rows) * groups;
  *bytes = static_cast<size_t>(units < kMostCtas ? units : kMostCtas) * 3 * (D / groups) * sizeof(float);
  return DL_OK;
}

int dl_block_norm_backward(int rows, int D, int groups, int in_dtype, const void* y, const float* post_weight,
                           const void* gate, const float* scale, const void* residual, const float* pre_weight, float eps,
                           const void* dout, const void* dnormed, void* dy, void* dgate, void* dresidual, float* dpost,
                           float* dscale, float* dpre, void* workspace, void* stream) {
  const int rc = check(rows, D, groups, in_dtype, y, scale, pre_weight, eps);
  if (rc != DL_OK) return rc;
  if ((dgate && !gate) || (dresidual && !residual) || (dpost && !post_weight) || (dscale && !scale) || (dpre && !pre_weight) || (dnormed && !pre_weight))
    return bad("gradient of a part that is not there");
  if (!ok_typed(in_dtype, {y, gate, residual, dout, dnormed, dy, dgate, dresidual}) ||
      !ok_typed(DL_F32, {post_weight, scale, pre_weight, dpost, dscale, dpre, workspace}))
    return bad("pointer not aligned to its element size");
  const bool sums = dpost || dscale || dpre;
  if (sums && rows > 0 && !workspace) return bad("parameter gradients need a workspace");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int n = D / groups;
  int ctas = 0;
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    NormArgs a{};
    a.y = y;
    a.gate = gate;
    a.residual = residual;
    a.post = post_weight;
    a.scale = scale;
    a.pre = pre_weight;
    a.dout = dout;
    a.dnormed = dnormed;
    a.dy = dy;
    a.dgate = dgate;
    a.dresidual = dresidual;
    a.partial = sums ? static_cast<float*>(workspace) : nullptr;
    a.groups = groups;
    a.n = n;
    a.rows = static_cast<long long>(rows) * groups;
    a.eps = eps;
    const Shape s = shape_of(n, in_dtype, wide_loads(n, in_dtype, {y, gate, residual, dout, dnormed, dy, dgate, dresidual},
                                                     {post_weight, scale, pre_weight}));
    a.tpr = s.tpr;
    ctas = backward_ctas(a.rows, s);
    e = run(a, s, ctas, in_dtype, true, st);
  }
  if (e == cudaSuccess && sums) {
    dl::norm_sums_kernel<<<dim3((n + 31) / 32, 3), dim3(32, 32), 0, st>>>(static_cast<const float*>(workspace), ctas, n, dpost,
                                                                         dscale, dpre);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? DL_OK : dl::launch_failed(e, "block norm backward launch");
}

}  // extern "C"
