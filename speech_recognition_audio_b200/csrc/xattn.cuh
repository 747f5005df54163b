// Shared by the cross-attention kernels: segment bounds, distributed shared
// memory reads, and the clusters that a device can hold.
#pragma once

#include "gemm2.cuh"
#include "kernels.h"
#include "splits.h"

namespace asr {

constexpr float kScaleLog2 = 0.125f * 1.4426950408889634f;  // log2(e) / sqrt(64)

struct Segment {
  int q0, lq, k0, lk;
  bool ok;
};

// Rows and states of segment `seg`; not ok (and reported) when its offsets
// leave the arrays or it is longer than the caller said.
__device__ __forceinline__ Segment load_segment(const XattnArgs& a, int seg, bool report) {
  Segment s;
  s.q0 = __ldg(a.cu_q + seg);
  s.k0 = __ldg(a.cu_k + seg);
  const int q1 = __ldg(a.cu_q + seg + 1), k1 = __ldg(a.cu_k + seg + 1);
  s.lq = q1 - s.q0;
  s.lk = k1 - s.k0;
  s.ok = s.q0 >= 0 && q1 >= s.q0 && q1 <= a.Tq && s.k0 >= 0 && k1 >= s.k0 && k1 <= a.Tk && s.lq <= a.max_q &&
         (a.width < 0 || s.lk <= a.width);
  if (!s.ok && report) atomicCAS(a.status, 0, DEV_BAD_SEGMENT);
  return s;
}

// The two halves of cluster_sync(), for the whole warp.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Maximum to subtract: 0 where no score is above -inf, so that
// exp(-inf - m) is 0 there and not NaN.
__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.f : m; }

// One output from its sum: an average of values of the type, so past f16's
// largest only because the probabilities were rounded for the product (a sum
// of theirs may exceed the one kept in 32 bits); infinities and NaN stay what
// they are.  bf16 reaches as far as the fp32 sums themselves.
template <int KIND>
__device__ __forceinline__ float average(float sum, float inv) {
  const float x = sum * inv;
  if constexpr (KIND == KIND_F16) return fabsf(x) < INFINITY ? fminf(fmaxf(x, -65504.f), 65504.f) : x;
  return x;
}

// Whether the current device can hold a cluster of 16 of these blocks, which
// is more than the portable size; asked once per device (`known` and `wide`
// are the caller's own masks of devices, one pair per kernel).
struct WideClusters {
  std::atomic<unsigned long long> known{0}, wide{0};
};
template <typename... KArgs>
bool holds_wide_cluster(void (*kernel)(KArgs...), int threads, size_t smem, WideClusters& seen) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (seen.known.load(std::memory_order_acquire) & bit)) return seen.wide.load(std::memory_order_relaxed) & bit;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 16;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  const bool ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                  cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0;
  if (!ok) cudaGetLastError();  // a refusal is an answer here, not an error of the call
  if (dev < 64) {
    if (ok) seen.wide.fetch_or(bit, std::memory_order_relaxed);
    seen.known.fetch_or(bit, std::memory_order_release);
  }
  return ok;
}

}  // namespace asr
