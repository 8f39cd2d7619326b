// clip.cu -- the global norm of many tensors' gradients, and clipping by it:
//
//   n = sqrt(sum over all tensors of g^2),  g' = g min(1, max_norm / (n + eps))
//
// Two kernels.  The first leaves one partial sum of squares per block, the
// second adds those (every block the same few hundred values in the same
// order, so all agree and nothing depends on timing) and scales.  The norm
// needs every value before the first one can be scaled, so the values are
// read twice unless they fit the L2: the second kernel walks the tensors
// from their end, where the first one has just been.
//
// HBM bounds both: 600 million bf16 values in 291 tensors take 175 us to square
// (6.9 TB/s) and 465 to scale (5.2 TB/s); 61 small tensors are two launches of
// 5 us behind 120 of the host, which reads every tensor's address, size and type.
//
// The tensors' addresses and sizes travel in the kernels' arguments: no
// table has to be copied to the device, and the calls can be captured.
#include "seq.h"

namespace fftgb {

constexpr int kClipThreads = 256;
constexpr int kClipBlocksPerSm = 3;
// A work item is 32 KB of one tensor: each thread loads its eight 16-byte
// vectors of it before it uses any.
constexpr int kClipVectors = 8;
constexpr long long kClipItemBytes = 16ll * kClipVectors * kClipThreads;
__host__ __device__ __forceinline__ int clip_size(int dtype) {
  return dtype == FFT_ELEM_F64 ? 8 : dtype == FFT_ELEM_F32 ? 4 : 2;
}

template <int N> struct ClipTable {
  const void *in[N];
  void *out[N];
  long long numel[N];
  long long first[N + 1];  // work items before the tensor
  signed char dtype[N];
  int count;
};
constexpr int kClipSmall = 72, kClipLarge = 960;  // 2.5 KB and 31.7 KB of kernel arguments
static_assert(sizeof(ClipTable<kClipLarge>) + 64 <= 32764, "kernel arguments");

template <int N> struct ClipItem {
  int t;
  long long begin, end;
  __device__ __forceinline__ ClipItem(const ClipTable<N> &tab, long long item) {
    int lo = 0, hi = tab.count - 1;  // the last tensor whose first item is not after `item`
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.first[mid] <= item) lo = mid;
      else hi = mid - 1;
    }
    t = lo;
    const long long each = kClipItemBytes / clip_size(tab.dtype[t]);
    begin = (item - tab.first[t]) * each;
    end = begin + each;
    if (end > tab.numel[t]) end = tab.numel[t];
  }
};

// Calls f(vector of 16 bytes, index) on the aligned vectors of [begin, end)
// and g(value, index) on what is left at both ends.
template <typename T, class F, class G>
__device__ __forceinline__ void walk(const T *p, long long begin, long long end, F f, G g) {
  constexpr int V = Vec16<T>::N;
  const long long skew = ((16 - ((uintptr_t)(p + begin) & 15u)) & 15u) / sizeof(T);
  long long vb = begin + skew;
  if (vb > end) vb = end;
  const int nv = (int)((end - vb) / V);
  const uint4 *q = reinterpret_cast<const uint4 *>(p + vb) + threadIdx.x;
  uint4 raw[kClipVectors];
  for (long long i = begin + threadIdx.x; i < vb; i += kClipThreads) g(p[i], i);
  for (long long i = vb + (long long)nv * V + threadIdx.x; i < end; i += kClipThreads) g(p[i], i);
#pragma unroll
  for (int u = 0; u < kClipVectors; ++u)
    raw[u] = (int)threadIdx.x + u * kClipThreads < nv ? q[u * kClipThreads]
                                                      : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int u = 0; u < kClipVectors; ++u)
    if ((int)threadIdx.x + u * kClipThreads < nv)
      f(raw[u], vb + (long long)(threadIdx.x + u * kClipThreads) * V);
}

// The squares of the same elements in fp64.
template <typename T>
__device__ __noinline__ double item_squares_fp64(const T *p, long long begin, long long end) {
  constexpr int V = Vec16<T>::N;
  double d = 0.0;
  walk<T>(
      p, begin, end,
      [&](uint4 w, long long) {
        typename Acc<T>::type f[V];
        unpack<T>(w, f);
        for (int i = 0; i < V; ++i) d += (double)f[i] * (double)f[i];
      },
      [&](T x, long long) {
        const double f = (double)to_acc(x);
        d += f * f;
      });
  return d;
}

// A thread's squares of an item: up to 64 of them in fp32, which is exact
// enough unless the sum overflows or is so small that squares were lost.
// Then, which no ordinary gradient reaches, they are taken again in fp64.
// (Adding to fp64 once per vector instead made the kernel wait for the few
// fp64 units.)
template <typename T>
__device__ __forceinline__ double item_squares(const T *p, long long begin, long long end) {
  constexpr int V = Vec16<T>::N;
  if constexpr (sizeof(T) < 8) {
    float s[2] = {0.0f, 0.0f};
    unsigned any = 0;
    walk<T>(
        p, begin, end,
        [&](uint4 w, long long) {
          any |= w.x | w.y | w.z | w.w;
          float f[V];
          unpack<T>(w, f);
#pragma unroll
          for (int i = 0; i < V; ++i) s[i & 1] = fmaf(f[i], f[i], s[i & 1]);
        },
        [&](T x, long long) {
          const float f = to_acc(x);
          any |= __float_as_uint(f);
          s[0] = fmaf(f, f, s[0]);
        });
    const float sum = s[0] + s[1];
    if (sum < 1e37f && (sum > 1e-24f || any == 0)) return (double)sum;
  }
  return item_squares_fp64(p, begin, end);
}

// The 16 bytes that start `skew` bytes (a multiple of 2) into eight words.
__device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, int skew) {
  unsigned w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (skew & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (skew & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (skew & 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements begin .. end of a tensor of n, times c.  Output vectors are
// aligned; where the input lies differently within its 16 bytes, a vector is
// cut from the two aligned ones it lies in (both inside the tensor).
template <typename T>
__device__ __forceinline__ void item_scale(const T *p, T *o, long long begin, long long end,
                                           long long n, typename Acc<T>::type c) {
  constexpr int V = Vec16<T>::N;
  const int skew = (int)(((uintptr_t)p - (uintptr_t)o) & 15u);
  long long vb = begin + (long long)(((16 - ((uintptr_t)(o + begin) & 15u)) & 15u) / sizeof(T));
  if (skew != 0 && vb * (long long)sizeof(T) < skew) vb += V;
  if (vb > end) vb = end;
  int nv = (int)((end - vb) / V);
  // the vector after the last one ends at or before the tensor's end
  const int room = (int)((n - vb) * (long long)sizeof(T) / 16) - 1;
  if (skew != 0 && nv > room) nv = room > 0 ? room : 0;
  for (long long i = begin + threadIdx.x; i < vb; i += kClipThreads)
    o[i] = from_acc<T>(to_acc(p[i]) * c);
  for (long long i = vb + (long long)nv * V + threadIdx.x; i < end; i += kClipThreads)
    o[i] = from_acc<T>(to_acc(p[i]) * c);
  const char *base = reinterpret_cast<const char *>(p + vb) - skew;
  const uint4 *q = reinterpret_cast<const uint4 *>(base) + threadIdx.x;
  uint4 *out = reinterpret_cast<uint4 *>(o + vb) + threadIdx.x;
  uint4 raw[kClipVectors];
#pragma unroll
  for (int u = 0; u < kClipVectors; ++u)
    raw[u] = (int)threadIdx.x + u * kClipThreads < nv ? q[u * kClipThreads] : make_uint4(0, 0, 0, 0);
  if (skew != 0) {
    uint4 next[kClipVectors];  // the neighbour's: in the cache
#pragma unroll
    for (int u = 0; u < kClipVectors; ++u)
      next[u] = (int)threadIdx.x + u * kClipThreads < nv ? q[u * kClipThreads + 1]
                                                         : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < kClipVectors; ++u) raw[u] = shifted(raw[u], next[u], skew);
  }
#pragma unroll
  for (int u = 0; u < kClipVectors; ++u)
    if ((int)threadIdx.x + u * kClipThreads < nv) {
      typename Acc<T>::type f[V];
      unpack<T>(raw[u], f);
#pragma unroll
      for (int k = 0; k < V; ++k) f[k] *= c;
      out[u * kClipThreads] = pack<T>(f);
    }
}

// Sum over the block in a fixed order, returned to every thread.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[kClipThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int k = 0; k < kClipThreads / 32; ++k) v += red[k];
  return v;
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipBlocksPerSm)
clip_squares_kernel(const __grid_constant__ ClipTable<N> tab, double *partial) {
  const long long items = tab.first[tab.count];
  double s = 0.0;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const ClipItem<N> w(tab, item);
    const void *p = tab.in[w.t];
    switch (tab.dtype[w.t]) {
      case FFT_ELEM_F32: s += item_squares(static_cast<const float *>(p), w.begin, w.end); break;
      case FFT_ELEM_F64: s += item_squares(static_cast<const double *>(p), w.begin, w.end); break;
      case FFT_ELEM_BF16:
        s += item_squares(static_cast<const __nv_bfloat16 *>(p), w.begin, w.end);
        break;
      default: s += item_squares(static_cast<const __half *>(p), w.begin, w.end);
    }
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipBlocksPerSm)
clip_scale_kernel(const __grid_constant__ ClipTable<N> tab, const double *partial, int parts,
                  double max_norm, double eps, float *norm) {
  double s = 0.0;
  for (int k = threadIdx.x; k < parts; k += kClipThreads) s += partial[k];
  const double n = sqrt(block_sum(s));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  // A norm that is NaN makes the factor NaN, an infinite one 0 (whatever the
  // bound); a quotient 0 / 0 clips nothing.
  const double f = max_norm / (n + eps);
  const double c = isinf(n) ? 0.0 : f < 1.0 || isnan(n) ? f : 1.0;
  const float cf = (float)c;
  const long long items = tab.first[tab.count];
  for (long long item = items - 1 - blockIdx.x; item >= 0; item -= gridDim.x) {
    const ClipItem<N> w(tab, item);
    const void *p = tab.in[w.t];
    void *o = tab.out[w.t];
    if (c == 1.0 && p == o) continue;  // in place and nothing to change
    switch (tab.dtype[w.t]) {
      case FFT_ELEM_F32:
        item_scale(static_cast<const float *>(p), static_cast<float *>(o), w.begin, w.end,
                   tab.numel[w.t], cf);
        break;
      case FFT_ELEM_F64:
        item_scale(static_cast<const double *>(p), static_cast<double *>(o), w.begin, w.end,
                   tab.numel[w.t], c);
        break;
      case FFT_ELEM_BF16:
        item_scale(static_cast<const __nv_bfloat16 *>(p), static_cast<__nv_bfloat16 *>(o),
                   w.begin, w.end,
                   tab.numel[w.t], cf);
        break;
      default:
        item_scale(static_cast<const __half *>(p), static_cast<__half *>(o), w.begin, w.end,
                   tab.numel[w.t], cf);
    }
  }
}

static int clip_grid(long long items) {
  const long long most = (long long)sm_count() * kClipBlocksPerSm;
  return (int)(items < most ? (items > 0 ? items : 1) : most);
}

size_t clip_workspace_bytes(long long count) {
  const long long launches = count > 0 ? (count + kClipLarge - 1) / kClipLarge : 1;
  return (size_t)launches * sm_count() * kClipBlocksPerSm * sizeof(double);
}

template <int N>
static void fill_table(ClipTable<N> &tab, long long begin, long long end, const void *const *in,
                       void *const *out, const int64_t *numel, const int *dtype) {
  tab.count = (int)(end - begin);
  long long items = 0;
  for (int k = 0; k < tab.count; ++k) {
    tab.in[k] = in[begin + k];
    tab.out[k] = out ? out[begin + k] : nullptr;
    tab.numel[k] = numel[begin + k];
    tab.dtype[k] = (signed char)dtype[begin + k];
    tab.first[k] = items;
    const long long each = kClipItemBytes / clip_size(tab.dtype[k]);
    items += (tab.numel[k] + each - 1) / each;
  }
  tab.first[tab.count] = items;
}

template <int N>
static cudaError_t clip_t(long long count, const void *const *in, void *const *out,
                          const int64_t *numel, const int *dtype, double max_norm, double eps,
                          float *norm, double *partial, cudaStream_t st) {
  ClipTable<N> tab;
  int parts = 0;
  for (long long b = 0; b < count || b == 0; b += N) {
    fill_table(tab, b, b + N < count ? b + N : count, in, out, numel, dtype);
    const int grid = clip_grid(tab.first[tab.count]);
    clip_squares_kernel<N><<<grid, kClipThreads, 0, st>>>(tab, partial + parts);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    parts += grid;
  }
  if (!out) {  // the norm alone
    tab.count = 0;
    tab.first[0] = 0;
    clip_scale_kernel<N><<<1, kClipThreads, 0, st>>>(tab, partial, parts, max_norm, eps, norm);
    return cudaGetLastError();
  }
  // Last tables first: their values were read last.
  const long long tables = count > 0 ? (count + N - 1) / N : 1;
  for (long long k = tables - 1; k >= 0; --k) {
    const long long b = k * N;
    if (k != tables - 1) fill_table(tab, b, b + N, in, out, numel, dtype);
    clip_scale_kernel<N><<<clip_grid(tab.first[tab.count]), kClipThreads, 0, st>>>(
        tab, partial, parts, max_norm, eps, k == 0 ? norm : nullptr);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_clip(long long count, const void *const *in, void *const *out,
                        const int64_t *numel, const int *dtype, double max_norm, double eps,
                        float *norm, void *workspace, cudaStream_t st) {
  double *partial = static_cast<double *>(workspace);
  return count <= kClipSmall ? clip_t<kClipSmall>(count, in, out, numel, dtype, max_norm, eps,
                                                  norm, partial, st)
                             : clip_t<kClipLarge>(count, in, out, numel, dtype, max_norm, eps,
                                                  norm, partial, st);
}

}  // namespace fftgb
