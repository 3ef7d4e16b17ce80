// Shared by the stateless operators (scan.cu, norm.cu, paged.cu): 16- and
// 32-bit element loads and stores as fp32, cluster barriers and remote shared
// memory stores, and the checks every entry point makes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "deltalog.h"
#include "ptx.cuh"

namespace dl {

int record_error(int code, const char* msg);  // api.cu: the last-error message of this thread

// N consecutive elements as they lie in memory, moved by one load or store of
// N * sizeof(T) bytes (a power of two up to 16; the address is that aligned).
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Streaming access (evict first): each element is read or written once.
template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load_stream(const T* p) {
  constexpr int BYTES = sizeof(T) * N;
  Pack<T, N> r;
  if constexpr (BYTES == 16) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    memcpy(&r, &u, 16);
  } else if constexpr (BYTES == 8) {
    const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
    memcpy(&r, &u, 8);
  } else if constexpr (BYTES == 4) {
    const unsigned u = __ldcs(reinterpret_cast<const unsigned*>(p));
    memcpy(&r, &u, 4);
  } else {
    const unsigned short u = __ldcs(reinterpret_cast<const unsigned short*>(p));
    memcpy(&r, &u, 2);
  }
  return r;
}

template <typename T, int N>
__device__ __forceinline__ void store_stream(T* p, const Pack<T, N>& r) {
  constexpr int BYTES = sizeof(T) * N;
  if constexpr (BYTES == 16) {
    uint4 u;
    memcpy(&u, &r, 16);
    __stcs(reinterpret_cast<uint4*>(p), u);
  } else if constexpr (BYTES == 8) {
    uint2 u;
    memcpy(&u, &r, 8);
    __stcs(reinterpret_cast<uint2*>(p), u);
  } else if constexpr (BYTES == 4) {
    unsigned u;
    memcpy(&u, &r, 4);
    __stcs(reinterpret_cast<unsigned*>(p), u);
  } else {
    unsigned short u;
    memcpy(&u, &r, 2);
    __stcs(reinterpret_cast<unsigned short*>(p), u);
  }
}

__device__ __forceinline__ void raise_error(int* err, int bit) {
  if (err) atomicOr(err, bit);
}

// Slot of row r under a slot map (null: the row itself); -1 for a row to skip,
// an index past the pool being reported by the thread with `tell`.
__device__ __forceinline__ int row_slot(const int* slot_idx, int slots, int r, int* err, bool tell) {
  if (!slot_idx) return r;
  const int raw = __ldg(slot_idx + r);
  if (raw < 0 || (raw & DL_SLOT_HOLD)) return -1;
  if (raw >= slots) {
    if (tell) raise_error(err, DL_DEVERR_SLOT_INDEX);
    return -1;
  }
  return raw;
}

// cp.async of 16 bytes of which the first `bytes` are read and the rest zeros.
__device__ __forceinline__ void copy_async16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(gmem_u64(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Thread-block cluster: this CTA's rank, a barrier of all its CTAs' threads
// (releases and acquires memory writes across the cluster), and the address of
// the same shared memory location in CTA `rank`.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote_smem(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// Only in a launch with cluster dimensions (an implicit cluster of one faults):
// floats into a CTA's shared memory, their bytes counted on the mbarrier
// `bar` of that CTA: data and signal in one, with no fence that would wait for
// this thread's earlier global stores (a cluster barrier in its place: 2.1 times
// the time of the 16385 x 1001 fp32 scan).
__device__ __forceinline__ void send_remote(uint32_t addr, uint32_t bar, float4 v) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr), "f"(v.x),
               "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void send_remote(uint32_t addr, uint32_t bar, float2 v) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(addr), "f"(v.x),
               "f"(v.y), "r"(bar)
               : "memory");
}

// Launch with cluster dimensions (n, 1, 1); n == 1 launches without clusters.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), dim3 grid, int block, size_t smem, cudaStream_t st, int n,
                           Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = n > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

inline bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline int launch_failed(cudaError_t e, const char* what) {
  cudaGetLastError();  // a refused launch leaves nothing behind for the caller's next check
  char buf[256];
  snprintf(buf, sizeof buf, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return record_error(DL_ERR_CUDA, buf);
}

}  // namespace dl
