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
// The tensors' addresses and sizes travel in the kernels' arguments: no
// table has to be copied to the device, and the calls can be captured.
#include "seq.h"

namespace fftgb {

constexpr int kClipThreads = 256;
constexpr int kClipBlocksPerSm = 3;
// Values per work item: enough that finding an item's tensor costs nothing,
// few enough that items spread evenly over the blocks.
constexpr long long kClipItem = 16384;

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

// Sum of the squares of N values.  Their fp32 sum is exact enough (N is
// small) unless it overflows or is so small that squares were lost: then,
// which no ordinary gradient reaches, the squares are taken in fp64.
template <int N> __device__ __forceinline__ double squares(const float (&v)[N]) {
  float s = 0.0f, m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s = fmaf(v[i], v[i], s);
    m = fmaxf(m, fabsf(v[i]));
  }
  if (s < 1e37f && (s > 1e-24f || m == 0.0f)) return (double)s;
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) d += (double)v[i] * (double)v[i];
  return d;
}

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
    begin = (item - tab.first[t]) * kClipItem;
    end = begin + kClipItem;
    if (end > tab.numel[t]) end = tab.numel[t];
  }
};

// Calls f(vector of 16 bytes, index) on the aligned vectors of [begin, end)
// and g(value, index) on what is left at both ends.
template <typename T, int UNROLL, class F, class G>
__device__ __forceinline__ void walk(const T *p, long long begin, long long end, F f, G g) {
  constexpr int V = Vec16<T>::N;
  const long long skew = ((16 - ((uintptr_t)(p + begin) & 15u)) & 15u) / sizeof(T);
  long long vb = begin + skew;
  if (vb > end) vb = end;
  const long long nv = (end - vb) / V;
  for (long long i = begin + threadIdx.x; i < vb; i += kClipThreads) g(p[i], i);
  for (long long i = vb + nv * V + threadIdx.x; i < end; i += kClipThreads) g(p[i], i);
  const uint4 *q = reinterpret_cast<const uint4 *>(p + vb);
  for (long long k = threadIdx.x; k < nv; k += (long long)UNROLL * kClipThreads) {
    uint4 raw[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (k + u * kClipThreads < nv) raw[u] = q[k + u * kClipThreads];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (k + u * kClipThreads < nv)
        f(*reinterpret_cast<const Vec16<T> *>(&raw[u]), vb + (k + u * kClipThreads) * V);
  }
}

template <typename T>
__device__ __forceinline__ double item_squares(const T *p, long long begin, long long end) {
  constexpr int V = Vec16<T>::N;
  double s = 0.0;
  walk<T, 4>(
      p, begin, end,
      [&](const Vec16<T> &x, long long) {
        if constexpr (sizeof(T) == 8) {
          for (int i = 0; i < V; ++i) s += x.v[i] * x.v[i];
        } else {
          float f[V];
#pragma unroll
          for (int i = 0; i < V; ++i) f[i] = to_acc(x.v[i]);
          s += squares(f);
        }
      },
      [&](T x, long long) {
        const double d = (double)to_acc(x);
        s += d * d;
      });
  return s;
}

template <typename T>
__device__ __forceinline__ void item_scale(const T *p, T *o, long long begin, long long end,
                                           typename Acc<T>::type c) {
  constexpr int V = Vec16<T>::N;
  const bool same = (((uintptr_t)p ^ (uintptr_t)o) & 15u) == 0;
  walk<T, 4>(
      p, begin, end,
      [&](Vec16<T> x, long long i) {
#pragma unroll
        for (int k = 0; k < V; ++k) x.v[k] = from_acc<T>(to_acc(x.v[k]) * c);
        if (same) {
          *reinterpret_cast<uint4 *>(o + i) = *reinterpret_cast<const uint4 *>(&x);
        } else {
#pragma unroll
          for (int k = 0; k < V; ++k) o[i + k] = x.v[k];
        }
      },
      [&](T x, long long i) { o[i] = from_acc<T>(to_acc(x) * c); });
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
  // NaN stays NaN (a comparison with it is false), and an infinite norm
  // scales by 0.
  const double f = max_norm / (n + eps);
  const double c = f > 1.0 ? 1.0 : f;
  const float cf = (float)c;
  const long long items = tab.first[tab.count];
  for (long long item = items - 1 - blockIdx.x; item >= 0; item -= gridDim.x) {
    const ClipItem<N> w(tab, item);
    const void *p = tab.in[w.t];
    void *o = tab.out[w.t];
    if (c == 1.0 && p == o) continue;  // in place and nothing to change
    switch (tab.dtype[w.t]) {
      case FFT_ELEM_F32:
        item_scale(static_cast<const float *>(p), static_cast<float *>(o), w.begin, w.end, cf);
        break;
      case FFT_ELEM_F64:
        item_scale(static_cast<const double *>(p), static_cast<double *>(o), w.begin, w.end, c);
        break;
      case FFT_ELEM_BF16:
        item_scale(static_cast<const __nv_bfloat16 *>(p), static_cast<__nv_bfloat16 *>(o),
                   w.begin, w.end, cf);
        break;
      default:
        item_scale(static_cast<const __half *>(p), static_cast<__half *>(o), w.begin, w.end, cf);
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
    items += (tab.numel[k] + kClipItem - 1) / kClipItem;
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
