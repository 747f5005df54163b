// Shared by the cross-attention kernels: segment bounds, distributed shared
// memory reads, and the launch of a grid whose clusters split the keys.
#pragma once

#include "gemm2.cuh"
#include "kernels.h"

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

// One output from its sum: an average of values of the type, so past the
// type's largest only because the probabilities were rounded for the product
// (a sum of theirs may exceed the one kept in 32 bits); infinities and NaN
// stay what they are.
template <int KIND>
__device__ __forceinline__ float average(float sum, float inv) {
  constexpr float top = KIND == KIND_F16 ? 65504.f : 3.3895313892515355e38f;
  const float x = sum * inv;
  return fabsf(x) < INFINITY ? fminf(fmaxf(x, -top), top) : x;
}

// Blocks a (segment, tile, head) is split into: a power of two, as long as the
// grid does not yet fill `fill` blocks and each block keeps at least `least`
// keys; up to `most` (8 is the portable cluster size, 16 needs allow_wide_clusters).
inline int pick_splits(long long blocks, int keys, int least, long long fill, int most = 8) {
  int s = 1;
  while (s < most && blocks * s < fill && keys >= 2 * s * least) s *= 2;
  return s;
}
// Lets a kernel be launched in clusters of 16, once per device.
template <typename... KArgs>
cudaError_t allow_wide_clusters(void (*kernel)(KArgs...), std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const unsigned long long bit = 1ull << (dev & 63);
  if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_relaxed) & bit))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace asr
