// What the operators over sequences (scan.cu, heads.cu, log_probs.cu, policy.cu)
// share.
#pragma once

#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "pieces.cuh"

namespace muon {

namespace {

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
// until at most N of the newest groups are in flight
template <int N> __device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n"
               "barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
// the address in block `rank` of the cluster of what is at p in this one
__device__ __forceinline__ uint32_t at_rank(const void* p, int rank) {
  uint32_t to;
  const uint32_t from = (uint32_t)__cvta_generic_to_shared(p);
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(from), "r"(rank));
  return to;
}
__device__ __forceinline__ void put_at(uint32_t to, const float4& f) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(f.x), "f"(f.y),
               "f"(f.z), "f"(f.w) : "memory");
}
__device__ __forceinline__ void put_at(uint32_t to, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
}
__device__ __forceinline__ void put_at(uint32_t to, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(v) : "memory");
}

// Launch in clusters of `cl` blocks
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), int64_t grid, int cl, int threads, size_t smem,
                           cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cl;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

inline bool off(const void* p, size_t es) { return reinterpret_cast<uintptr_t>(p) % es != 0; }
template <typename... P> bool any_off(size_t es, const P*... p) { return (off(p, es) || ...); }

// f(value of the element type)
template <typename F> auto by_type(int dtype, F f) {
  if (dtype == MUON_BF16) return f(__nv_bfloat16());
  return f(float());
}
inline size_t size_of(int dtype) { return dtype == MUON_BF16 ? 2 : 4; }
inline bool known(int dtype) { return dtype == MUON_BF16 || dtype == MUON_F32; }

}  // namespace

}  // namespace muon
