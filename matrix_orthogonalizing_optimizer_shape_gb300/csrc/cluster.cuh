// Thread-block clusters: barriers and stores to another block's shared memory.
#pragma once

#include <cstdint>

namespace dion3 {
namespace cl {

__device__ __forceinline__ void arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ int rank() {
  int r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int size() {
  int r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Address in block `rank`'s shared memory of what lies at `shared` in this one's.
__device__ __forceinline__ uint32_t peer(const void* shared, int rank) {
  const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(shared));
  uint32_t remote;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  return remote;
}
__device__ __forceinline__ void store(uint32_t at, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
// Counts its bytes on the mbarrier `bar` of the same block when they are there.
__device__ __forceinline__ void store_async(uint32_t at, float2 v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at), "f"(v.x),
               "f"(v.y), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void store(uint32_t at, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

}  // namespace cl
}  // namespace dion3
