// What the kernels of the head norm and of the embedding use beside cluster.cuh:
// attributes set once a device, and loads from a peer's shared memory.
#pragma once

#include <atomic>

#include "cluster.cuh"

namespace rmsn {

// Lets KERNEL use `bytes` of dynamic shared memory, and clusters of more than 8
// CTAs, once a device.
template <auto KERNEL>
cudaError_t allow_launch(int dev, size_t bytes) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const void* kern = reinterpret_cast<const void*>(KERNEL);
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// The word at `local` in the shared memory of CTA `peer` of the cluster.
__device__ __forceinline__ uint32_t ld_peer(const void* local, uint32_t peer) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
  uint32_t remote, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(a), "r"(peer));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

}  // namespace rmsn
