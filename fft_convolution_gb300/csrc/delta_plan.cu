// delta_plan.cu -- where the chunks of packed sequences lie: the sequences'
// first rows and the number of chunks before each, from the caller's offsets
// on the device (the host never sees them).  Rows before the first sequence and
// after the last one, which nothing else writes, are cleared in the same launch.
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

constexpr int kClearBlocks = 64;

// Zeros, of elements of 2 bytes or more.
__device__ __forceinline__ void clear_bytes(char *p, long long bytes, int thread, int threads) {
  if (bytes <= 0) return;
  long long head = (16 - ((uintptr_t)p & 15)) & 15;
  if (head > bytes) head = bytes;
  const long long words = (bytes - head) >> 4, done = head + (words << 4);
  for (long long i = 2ll * thread; i < head; i += 2ll * threads)
    *reinterpret_cast<uint16_t *>(p + i) = 0;
  for (long long i = thread; i < words; i += threads)
    reinterpret_cast<uint4 *>(p + head)[i] = make_uint4(0, 0, 0, 0);
  for (long long i = done + 2ll * thread; i < bytes; i += 2ll * threads)
    *reinterpret_cast<uint16_t *>(p + i) = 0;
}

// Offsets that descend or leave the rows are raised or cut to the nearest
// that do not: every later access stays within the arrays.
__global__ void __launch_bounds__(1024)
delta_plan_kernel(const int *offsets, int batch, int tokens, int *row0, int *chunk0,
                  const DeltaClear clear) {
  __shared__ int sums[32];
  if (blockIdx.x > 0) {
    int last = 0;  // the row after the last sequence
    for (int i = threadIdx.x; i <= batch; i += 1024) last = max(last, min(offsets[i], tokens));
    last = __reduce_max_sync(0xffffffffu, last);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = last;
    __syncthreads();
    last = __reduce_max_sync(0xffffffffu, sums[threadIdx.x & 31]);
    const int first = max(0, min(offsets[0], tokens));
    const int thread = (blockIdx.x - 1) * 1024 + threadIdx.x, threads = (gridDim.x - 1) * 1024;
    for (int k = 0; k < clear.count; ++k) {
      char *p = static_cast<char *>(clear.p[k]);
      const long long bytes = clear.row_bytes[k];
      clear_bytes(p, first * bytes, thread, threads);
      clear_bytes(p + last * bytes, (tokens - last) * bytes, thread, threads);
    }
    return;
  }
  if (!row0) return;
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
                              int *chunk0, const DeltaClear &clear, cudaStream_t st) {
  delta_plan_kernel<<<clear.count > 0 ? 1 + kClearBlocks : 1, 1024, 0, st>>>(
      offsets, (int)batch, (int)tokens, row0, chunk0, clear);
  return cudaGetLastError();
}

DeltaClear delta_clear(const DeltaArgs &a, const DeltaGradArgs *g, size_t elem) {
  DeltaClear c{};
  if (!a.clear) return c;
  auto add = [&](void *p, size_t row_bytes) {
    if (!p) return;
    c.p[c.count] = p;
    c.row_bytes[c.count++] = (long long)row_bytes;
  };
  const size_t v = (size_t)a.vheads * a.dv * elem, k = (size_t)a.kheads * a.dk * elem;
  add(a.o, v);
  if (g) {
    add(g->dq, k);
    add(g->dk, k);
    add(g->dv, v);
    add(g->dg, (size_t)a.vheads * 4);
    add(g->dbeta, (size_t)a.vheads * 4);
  }
  return c;
}

size_t delta_workspace_bytes(const DeltaArgs &a, bool packed) {
  return DeltaLayout(a, packed, false).bytes;
}
size_t delta_grad_workspace_bytes(const DeltaArgs &a, bool packed) {
  return DeltaLayout(a, packed, true).bytes;
}

}  // namespace fftgb
