// delta_plan.cu -- where the chunks of packed sequences lie: the sequences'
// first rows and the number of chunks before each, from the caller's offsets
// on the device (the host never sees them).
#include "delta.cuh"

namespace fftgb {

// Inclusive scan over 1024 threads of f(a, b) from left to right, starting
// from `carry`, which becomes the last value.
template <class F>
__device__ __forceinline__ int block_scan(int v, int *sums, int &carry, int identity, F f) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = f(t, v);
  }
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s = f(t, s);
    }
    sums[lane] = s;
  }
  __syncthreads();
  v = f(f(carry, warp > 0 ? sums[warp - 1] : identity), v);
  carry = f(carry, sums[31]);
  __syncthreads();
  return v;
}

// Offsets that descend or leave the rows are raised or cut to the nearest
// that do not: every later access stays within the arrays.
__global__ void __launch_bounds__(1024)
delta_plan_kernel(const int *offsets, int batch, int tokens, int *row0, int *chunk0) {
  __shared__ int sums[32];
  int carry = 0;
  for (int base = 0; base <= batch; base += 1024) {
    const int i = base + threadIdx.x;
    int v = i <= batch ? offsets[i] : 0;
    v = v < 0 ? 0 : v > tokens ? tokens : v;
    v = block_scan(v, sums, carry, 0, [](int x, int y) { return x > y ? x : y; });
    if (i <= batch) row0[i] = v;
  }
  __syncthreads();
  carry = 0;
  if (threadIdx.x == 0) chunk0[0] = 0;
  for (int base = 0; base < batch; base += 1024) {
    const int i = base + threadIdx.x;
    const int n = i < batch ? (row0[i + 1] - row0[i] + kChunk - 1) / kChunk : 0;
    const int s = block_scan(n, sums, carry, 0, [](int x, int y) { return x + y; });
    if (i < batch) chunk0[i + 1] = s;
  }
}

cudaError_t launch_delta_plan(const int *offsets, long long batch, long long tokens, int *row0,
                              int *chunk0, cudaStream_t st) {
  delta_plan_kernel<<<1, 1024, 0, st>>>(offsets, (int)batch, (int)tokens, row0, chunk0);
  return cudaGetLastError();
}

size_t delta_workspace_bytes(const DeltaArgs &a, bool packed) {
  return DeltaLayout(a, packed, false).bytes;
}
size_t delta_grad_workspace_bytes(const DeltaArgs &a, bool packed) {
  return DeltaLayout(a, packed, true).bytes;
}

}  // namespace fftgb
