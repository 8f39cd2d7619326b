// cluster.cuh -- thread-block clusters as the kernels of sequence models use
// them: barriers, and shared memory of the other blocks.
#pragma once

#include <stdint.h>

#include "tcgen05.cuh"

namespace fftgb {

__device__ __forceinline__ uint32_t block_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of the cluster arrives; what it has written before (shared
// memory of any block, global memory) is seen by those that have waited.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// The address of the same shared variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t peer_load(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// Writes 16 bytes into another block's shared memory and counts them at its
// barrier: no fence, so stores to global memory under way hold nothing up.
__device__ __forceinline__ void peer_send(uint32_t addr, float4 v, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, "
      "[%5];" ::"r"(addr),
      "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
      : "memory");
}

// Whether the phase has completed, other blocks' writes before it seen.
__device__ __forceinline__ bool poll_cluster(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// A wait for it that ends after `limit` clocks, or when `failed` (shared memory) says
// that another of the block's has; `status`: the device status word.
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, volatile int *failed,
                                             int *status, long long limit) {
  if (poll_cluster(bar, parity)) return true;
  const long long t0 = clock64();
#pragma unroll 1
  for (uint32_t it = 0; it < (1u << 24); ++it) {
    if (poll_cluster(bar, parity)) return true;
    if (*failed || clock64() - t0 > limit) break;
  }
  *failed = 1;
  atomicExch(status, 1);  // kDeviceErrorTimeout
  return false;
}

// How a block that has given up leaves: its own copies, which take microseconds, are waited for,
// some milliseconds at most (a barrier that has been given up may never complete).
__device__ __forceinline__ void let_land(uint64_t *bar, uint32_t parity) {
#pragma unroll 1
  for (int it = 0; it < 4096 && !bar_poll(bar, parity); ++it) __nanosleep(2048);
}
// And what other blocks have sent it, which it does not count any more, gets about 60 us.
__device__ __forceinline__ void linger() {
#pragma unroll 1
  for (int it = 0; it < 64; ++it) __nanosleep(1024);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

}  // namespace fftgb
