// layer_norm.cuh -- layer normalisation of rows, forward and backward.
//
//   forward   mu = mean(x), r = (mean((x - mu)^2) + eps)^-1/2,
//             y = (x - mu) r w + b
//   backward  xh = (x - mu) r, d = dy w,
//             dx = r (d - mean(d) - xh mean(d xh)),
//             dw = sum over rows of dy xh, db = sum over rows of dy
//
// Both directions read and write every row once, so HBM bounds them.  A row
// stays in the registers of the TPR threads that share it (EPT elements
// each): the variance is taken about the mean in a second pass over
// registers, not from a difference of two large sums.  Blocks are persistent
// and walk the rows; a thread keeps the same columns throughout, so w and b
// are read once per block, and the sums of dw and db over the block's rows
// stay in registers: one row of partial sums per block goes to HBM, and a
// second kernel adds those in a fixed order (no atomics, so the result does
// not depend on timing).  All sums are fp32 (fp64 rows: fp64).
#pragma once

#include "seq.h"
#include "tcgen05.cuh"

namespace fftgb {

// Sum over the TPR threads that share a row, returned to all of them.  `red`
// holds two sets of TPR / 32 values and is used alternately, which saves the
// barrier between reading one sum and writing the next.
template <int TPR, typename A>
__device__ __forceinline__ A row_sum(A v, A *red, int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    A *r = red + turn * W;
    if ((threadIdx.x & 31) == 0) r[(threadIdx.x % TPR) >> 5] = v;
    __syncthreads();
    v = r[threadIdx.x & (W - 1)];
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    turn ^= 1;
  }
  return v;
}

// Mean of a row and the sum of squares about it with one barrier: a warp takes
// both of its own elements (the squares about its own mean, from registers),
// and the warps' are joined by M = sum over warps of M_w + n_w (mean_w - mean)^2.
// n: this warp's elements; elements beyond the row hold 0.
template <int TPR, int EPT, class Inside>
__device__ __forceinline__ float2 row_moments(const float (&f)[EPT], float n, float inv_dim,
                                              float4 *red, int &turn, Inside inside) {
  float s = 0.0f, m = 0.0f;
#pragma unroll
  for (int e = 0; e < EPT; ++e) s += f[e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float mean_w = n > 0.0f ? s / n : 0.0f;
#pragma unroll
  for (int e = 0; e < EPT; ++e) {
    const float d = f[e] - mean_w;
    if (inside(e)) m = fmaf(d, d, m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
  if constexpr (TPR == 32) {
    return make_float2(mean_w, m);
  } else {
    constexpr int W = TPR / 32;
    float4 *r = red + turn * W;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = make_float4(s, m, mean_w, n);
    __syncthreads();
    turn ^= 1;
    const float4 w = r[threadIdx.x & (W - 1)];
    s = w.x;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mean = s * inv_dim, d = w.z - mean;
    m = fmaf(w.w * d, d, w.y);
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    return make_float2(mean, m);
  }
}

// Both sums of a row of the backward pass in one round.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2 *red, int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    float2 *r = red + turn * W;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const float2 t = r[threadIdx.x & (W - 1)];
    a = t.x;
    b = t.y;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    turn ^= 1;
  }
  return make_float2(a, b);
}
// The same of two rows.  Lanes halve the values they carry at each step (one of
// four is left after two), then each sums one of them over the warps.
template <int TPR>
__device__ __forceinline__ float4 row_sum4(float4 v, float4 *red, int &turn) {
  const int lane = threadIdx.x & 31;
  const bool b4 = lane & 16, b3 = lane & 8;
  auto trade = [](float keep, float give, int o) {
    return keep + __shfl_xor_sync(0xffffffffu, give, o);
  };
  const float x = trade(b4 ? v.z : v.x, b4 ? v.x : v.z, 16);
  const float y = trade(b4 ? v.w : v.y, b4 ? v.y : v.w, 16);
  float s = trade(b3 ? y : x, b3 ? x : y, 8);  // value 2 b4 + b3
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  int from = 8;  // lanes from one value to the next
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    float *r = reinterpret_cast<float *>(red + turn * W);
    if ((lane & 7) == 0) r[(threadIdx.x >> 5) * 4 + (lane >> 3)] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 4 * W; k += 32)
      if (k + lane < 4 * W) s += r[k + lane];
#pragma unroll
    for (int o = 4; o < (4 * W < 32 ? 4 * W : 32); o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    turn ^= 1;
    from = 1;
  }
  v.x = __shfl_sync(0xffffffffu, s, 0);
  v.y = __shfl_sync(0xffffffffu, s, from);
  v.z = __shfl_sync(0xffffffffu, s, 2 * from);
  v.w = __shfl_sync(0xffffffffu, s, 3 * from);
  return v;
}

// Column of a thread's element e: 16-byte vectors (VEC), or single elements
// at a stride of TPR where the rows are not 16-byte aligned.
template <typename T, int TPR, bool VEC>
__device__ __forceinline__ int column(int t, int e) {
  constexpr int N = Vec16<T>::N;
  if constexpr (VEC) return ((e / N) * TPR + t) * N + e % N;
  return e * TPR + t;
}

// A thread's part of a row as loaded: whole 16-byte words where the rows allow
// it (16-bit elements then stay two to a register).
template <typename T, int TPR, int EPT, bool VEC> struct RowRegs;
template <typename T, int TPR, int EPT> struct RowRegs<T, TPR, EPT, true> {
  static constexpr int N = Vec16<T>::N;
  uint4 raw[EPT / N];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < EPT / N; ++k) raw[k] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const T *row, int t, int dim) {
#pragma unroll
    for (int k = 0; k < EPT / N; ++k) {
      const int c = (k * TPR + t) * N;
      raw[k] = c < dim ? __ldcs(reinterpret_cast<const uint4 *>(row + c)) : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void get(float (&f)[EPT]) const {
#pragma unroll
    for (int k = 0; k < EPT / N; ++k) {
      float g[N];
      unpack<T>(raw[k], g);
#pragma unroll
      for (int i = 0; i < N; ++i) f[k * N + i] = g[i];
    }
  }
  static __device__ __forceinline__ void store(T *row, const float (&f)[EPT], int t, int dim) {
#pragma unroll
    for (int k = 0; k < EPT / N; ++k) {
      const int c = (k * TPR + t) * N;
      float g[N];
#pragma unroll
      for (int i = 0; i < N; ++i) g[i] = f[k * N + i];
      if (c < dim) *reinterpret_cast<uint4 *>(row + c) = pack<T>(g);
    }
  }
};
template <typename T, int TPR, int EPT> struct RowRegs<T, TPR, EPT, false> {
  T v[EPT];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < EPT; ++e) v[e] = from_acc<T>(0.0f);
  }
  __device__ __forceinline__ void load(const T *row, int t, int dim) {
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      const int c = e * TPR + t;
      v[e] = c < dim ? row[c] : from_acc<T>(0.0f);
    }
  }
  __device__ __forceinline__ void get(float (&f)[EPT]) const {
#pragma unroll
    for (int e = 0; e < EPT; ++e) f[e] = to_acc(v[e]);
  }
  static __device__ __forceinline__ void store(T *row, const float (&f)[EPT], int t, int dim) {
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      const int c = e * TPR + t;
      if (c < dim) row[c] = from_acc<T>(f[e]);
    }
  }
};
// Rows under way per thread: each is loaded that many rounds before it is
// used, into registers of its own (moving a row would wait for it).
template <typename T, bool VEC, int MOST> constexpr int kNormDepth = VEC && sizeof(T) == 2 ? MOST : 1;

// Rows of one warp share blocks of eight; other rows have a block each.
template <int TPR> struct NormBlock {
  static constexpr int THREADS = TPR == 32 ? 256 : TPR;
  static constexpr int GROUPS = THREADS / TPR;
  // Blocks per multiprocessor: 1024 threads, which leaves them 64 registers;
  // half of that for rows of one warp, which hold more and wait for no one.
  static constexpr int BLOCKS = TPR == 32 ? 2 : THREADS >= 1024 ? 1 : 1024 / THREADS;
};

template <typename T, int TPR, int EPT, bool VEC>
__global__ void __launch_bounds__(NormBlock<TPR>::THREADS, NormBlock<TPR>::BLOCKS)
layer_norm_kernel(const LayerNormArgs a) {
  constexpr int G = NormBlock<TPR>::GROUPS;
  __shared__ float4 red[2 * 32];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const T *x = static_cast<const T *>(a.x);
  T *y = static_cast<T *>(a.y);
  float w[EPT], b[EPT], n = 0.0f;
#pragma unroll
  for (int e = 0; e < EPT; ++e) {
    const int c = column<T, TPR, VEC>(t, e);
    w[e] = a.w && c < a.dim ? load_any(a.w, a.wtype, c) : 1.0f;
    b[e] = a.b && c < a.dim ? load_any(a.b, a.wtype, c) : 0.0f;
    if (c < a.dim) n += 1.0f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  const float inv = 1.0f / (float)a.dim;
  int turn = 0;
  const long long step = (long long)gridDim.x * G;
  long long row = (long long)blockIdx.x * G + grp;
  constexpr int DEPTH = kNormDepth<T, VEC, 3>;
  RowRegs<T, TPR, EPT, VEC> buf[DEPTH];
#pragma unroll
  for (int k = 0; k < DEPTH; ++k)
    if (row + k * step < a.rows) buf[k].load(x + (row + k * step) * a.ldx, t, a.dim);
  // The row groups of a block share no barrier (a group of several warps is
  // a whole block), so each may end its loop on its own.
  while (row < a.rows) {
#pragma unroll
    for (int k = 0; k < DEPTH; ++k, row += step) {
      if (row >= a.rows) break;
      float f[EPT];
      buf[k].get(f);
      if (row + DEPTH * step < a.rows) buf[k].load(x + (row + DEPTH * step) * a.ldx, t, a.dim);
      const float2 m = row_moments<TPR, EPT>(
          f, n, inv, red, turn, [&](int e) { return column<T, TPR, VEC>(t, e) < a.dim; });
      const float mu = m.x, r = 1.0f / sqrtf(m.y * inv + (float)a.eps);
#pragma unroll
      for (int e = 0; e < EPT; ++e) f[e] = (f[e] - mu) * r * w[e] + b[e];
      RowRegs<T, TPR, EPT, VEC>::store(y + row * a.ldy, f, t, a.dim);
      if (t == 0) {
        if (a.mean) static_cast<float *>(a.mean)[row] = mu;
        if (a.rstd) static_cast<float *>(a.rstd)[row] = r;
      }
    }
  }
}

// Rows that W = 1 or 2 warps hold whole (NV 16-byte words per lane): no barrier
// at all, or one between two warps.  While a row is worked on, each lane copies
// its words of the next one to shared memory, where nobody else reads them.  w
// and b lie there in fp32.  16384 x 4096 bf16: two warps per row 46 us, 87% of
// the copy rate (51 without the copies ahead); one warp with 16 words per lane
// spills, 60; a block per row waits for its barrier most of the time, 70.
template <typename T, int NV, int W>
__global__ void __launch_bounds__(256, 2) layer_norm_warp_kernel(const LayerNormArgs a) {
  extern __shared__ float wb[];  // w, then b
  __shared__ float2 red[2][8];
  constexpr int N = Vec16<T>::N;
  const int t = threadIdx.x % (32 * W), warp = threadIdx.x >> 5;
  float *ws = wb, *bs = wb + a.dim;
  for (int c = threadIdx.x; c < a.dim; c += 256) {
    ws[c] = a.w ? load_any(a.w, a.wtype, c) : 1.0f;
    bs[c] = a.b ? load_any(a.b, a.wtype, c) : 0.0f;
  }
  __syncthreads();
  const float inv = 1.0f / (float)a.dim;
  // elements of a row that this warp has
  float mine = (float)a.dim;
  if constexpr (W > 1) {
    const int words = (int)(a.dim / N), rounds = words / (32 * W), rest = words % (32 * W) - (t & ~31);
    mine = (float)((rounds * 32 + (rest < 0 ? 0 : rest > 32 ? 32 : rest)) * N);
  }
  int turn = 0;
  const long long step = (long long)gridDim.x * (8 / W);
  // The next row's words, each lane its own.
  uint4 *mine_words = reinterpret_cast<uint4 *>(wb + 2 * a.dim) + threadIdx.x;
  auto fetch = [&](long long row) {
    const T *x = static_cast<const T *>(a.x) + row * a.ldx + t * N;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if ((k * 32 * W + t) * N < a.dim) copy16(smem_u32(mine_words + k * 256), x + k * 32 * W * N);
  };
  long long row = (long long)blockIdx.x * (8 / W) + warp / W;
  if (row < a.rows) fetch(row);
  for (; row < a.rows; row += step) {
    T *y = static_cast<T *>(a.y) + row * a.ldy;
    uint4 raw[NV];
    copy_wait_all();
#pragma unroll
    for (int k = 0; k < NV; ++k)
      raw[k] = (k * 32 * W + t) * N < a.dim ? mine_words[k * 256] : make_uint4(0, 0, 0, 0);
    // Three walks over the registers, two values per instruction.
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float f[N];
      unpack<T>(raw[k], f);
#pragma unroll
      for (int i = 0; i < N; i += 2) s = fma2(make_float2(f[i], f[i + 1]), both(1.0f), s);
    }
    s.x += s.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
    float mu = W == 1 ? s.x * inv : mine > 0.0f ? s.x / mine : 0.0f;
    if (row + step < a.rows) fetch(row + step);  // (every word has been used)
    s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float f[N];
      unpack<T>(raw[k], f);
      if ((k * 32 * W + t) * N < a.dim) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const float2 d = fma2(both(-mu), both(1.0f), make_float2(f[i], f[i + 1]));
          s = fma2(d, d, s);
        }
      }
    }
    s.x += s.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
    if constexpr (W > 1) {
      // both warps' squares about their own means, joined (row_moments)
      const float own = mu, n = mine, m = (float)a.dim - mine;
      if ((t & 31) == 0) red[turn][warp] = make_float2(own, s.x);
      asm volatile("bar.sync %0, 64;" ::"r"(1 + warp / 2) : "memory");
      const float2 o = red[turn][warp ^ 1];
      turn ^= 1;
      mu = (own * n + o.x * m) * inv;
      const float d = own - mu, e = o.x - mu;
      s.x = (s.x + o.y) + (n * d * d + m * e * e);
    }
    const float r = 1.0f / sqrtf(s.x * inv + (float)a.eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * 32 * W + t) * N;
      if (c < a.dim) {
        float f[N];
        unpack<T>(raw[k], f);
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const float4 w = *reinterpret_cast<const float4 *>(ws + c + i);
          const float4 b = *reinterpret_cast<const float4 *>(bs + c + i);
#pragma unroll
          for (int h = 0; h < 4; h += 2) {
            const float2 d = mul2(fma2(both(-mu), both(1.0f), make_float2(f[i + h], f[i + h + 1])),
                                  both(r));
            const float2 o = fma2(d, h ? make_float2(w.z, w.w) : make_float2(w.x, w.y),
                                  h ? make_float2(b.z, b.w) : make_float2(b.x, b.y));
            f[i + h] = o.x;
            f[i + h + 1] = o.y;
          }
        }
        *reinterpret_cast<uint4 *>(y + c) = pack<T>(f);
      }
    }
    if (t == 0) {
      if (a.mean) static_cast<float *>(a.mean)[row] = mu;
      if (a.rstd) static_cast<float *>(a.rstd)[row] = r;
    }
  }
}
template <typename T, int NV = 1, int W = 1>
cudaError_t layer_norm_warp(const LayerNormArgs &a, cudaStream_t st) {
  if constexpr (NV < 8) {
    if (a.dim > NV * 32 * Vec16<T>::N) return layer_norm_warp<T, 2 * NV, 1>(a, st);
  } else if constexpr (W == 1) {
    if (a.dim > NV * 32 * Vec16<T>::N) return layer_norm_warp<T, NV, 2>(a, st);
  }
  const long long blocks = (a.rows * W + 7) / 8, most = 2ll * sm_count();
  constexpr size_t words = 256 * NV * 16;
  static DeviceOnce once;
  const cudaError_t e = smem_limit_once((const void *)layer_norm_warp_kernel<T, NV, W>,
                                        words + 2 * W * NV * 32 * Vec16<T>::N * sizeof(float), once);
  if (e != cudaSuccess) return e;
  layer_norm_warp_kernel<T, NV, W><<<(int)(blocks < most ? blocks : most), 256,
                                     words + 2 * a.dim * sizeof(float), st>>>(a);
  return cudaGetLastError();
}

// Rows shared by several warps, on 16-byte boundaries, are copied to shared
// memory ahead: 64 bytes per thread and round, three rounds, 192 KB per SM
// (16384 x 4096 bf16, loaded into registers for the next round only: 112 us; copied
// 106; 16-bit rows read from there again for dx, which spares the registers that
// spilled, 97; fewer shuffles in the rows' sums, 91).
constexpr int kNormStages = 3, kNormRoundBytes = 64;
template <int TPR, bool VEC> __host__ __device__ constexpr bool norm_ring() { return VEC && TPR > 32; }
template <int TPR, bool VEC> constexpr size_t norm_grad_smem() {
  return norm_ring<TPR, VEC>() ? (size_t)kNormStages * kNormRoundBytes * NormBlock<TPR>::THREADS : 0;
}

// 16-bit rows: two per round share one barrier (fp32 rows would not fit the
// registers).
template <typename T, int TPR, int EPT, bool VEC>
__global__ void __launch_bounds__(NormBlock<TPR>::THREADS, NormBlock<TPR>::BLOCKS)
layer_norm_grad_kernel(const LayerNormGradArgs a) {
  constexpr int G = NormBlock<TPR>::GROUPS;
  __shared__ float4 red[2 * 32];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);
  const float *mean = static_cast<const float *>(a.mean);
  const float *rstd = static_cast<const float *>(a.rstd);
  T *dx = static_cast<T *>(a.dx);
  // Two elements per instruction: the fp32 rows of 3001 elements, without vector
  // loads, went from 42 to 39 us.
  constexpr int PAIRS = EPT / 2;
  float2 w[PAIRS], dw[PAIRS], db[PAIRS];
#pragma unroll
  for (int e = 0; e < PAIRS; ++e) {
    auto weight = [&](int c) { return a.w && c < a.dim ? load_any(a.w, a.wtype, c) : 1.0f; };
    w[e] = make_float2(weight(column<T, TPR, VEC>(t, 2 * e)), weight(column<T, TPR, VEC>(t, 2 * e + 1)));
    dw[e] = db[e] = make_float2(0.0f, 0.0f);
  }
  constexpr int ROWS = VEC && sizeof(T) == 2 ? 2 : 1;
  constexpr bool RING = norm_ring<TPR, VEC>();
  const float inv = 1.0f / (float)a.dim;
  int turn = 0;
  const long long step = (long long)gridDim.x * G;
  long long row = (long long)blockIdx.x * G + grp;
  RowRegs<T, TPR, EPT, VEC> xb[ROWS], gb[ROWS];
  float mu[ROWS], r[ROWS];
  auto load = [&](int k, long long at) {
    if (at < a.rows) {
      xb[k].load(x + at * a.ldx, t, a.dim);
      gb[k].load(dy + at * a.lddy, t, a.dim);
      mu[k] = mean[at];
      r[k] = rstd[at];
    } else {
      xb[k].zero();
      gb[k].zero();
      mu[k] = r[k] = 0.0f;  // a row that adds nothing
    }
  };
  // RING: a thread's words of the rows ahead, nobody else reads them.
  constexpr int WORDS = VEC ? EPT / Vec16<T>::N : 1;
  extern __shared__ uint4 norm_ring_words[];
  uint4 *mine = norm_ring_words + threadIdx.x;
  auto word = [&](int stage, int k, int which, int j) {
    return mine + (((stage * ROWS + k) * 2 + which) * WORDS + j) * NormBlock<TPR>::THREADS;
  };
  auto fetch = [&](int stage, long long first) {
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const long long at = first + k * step;
      if (at < a.rows)
#pragma unroll
        for (int j = 0; j < WORDS; ++j) {
          const int c = (j * TPR + t) * Vec16<T>::N;
          if (c < a.dim) {
            copy16(smem_u32(word(stage, k, 0, j)), x + at * a.ldx + c);
            copy16(smem_u32(word(stage, k, 1, j)), dy + at * a.lddy + c);
          }
        }
    }
    copy_group();
  };
  float next_mu[ROWS], next_r[ROWS];
  auto moments = [&](int k, long long at) {
    next_mu[k] = at < a.rows ? mean[at] : 0.0f;
    next_r[k] = at < a.rows ? rstd[at] : 0.0f;
  };
  int stage = 0;
  auto take = [&](int k) {
    if constexpr (RING) {
#pragma unroll
      for (int j = 0; j < WORDS; ++j) {
        const bool there = row + k * step < a.rows && (j * TPR + t) * Vec16<T>::N < a.dim;
        xb[k].raw[j] = there ? *word(stage, k, 0, j) : make_uint4(0, 0, 0, 0);
        gb[k].raw[j] = there ? *word(stage, k, 1, j) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  if constexpr (RING) {
#pragma unroll
    for (int i = 0; i < kNormStages; ++i) fetch(i, row + i * ROWS * step);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) moments(k, row + k * step);
  } else if (row < a.rows) {
#pragma unroll
    for (int k = 0; k < ROWS; ++k) load(k, row + k * step);
  }
  for (; row < a.rows; row += ROWS * step) {
    if constexpr (RING) {
      copy_wait<kNormStages - 1>();
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        mu[k] = next_mu[k];
        r[k] = next_r[k];
        moments(k, row + (k + ROWS) * step);
        take(k);
      }
    }
    float s[4];
    const float2 one = both(1.0f);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      float xh[EPT], g[EPT];
      xb[k].get(xh);
      gb[k].get(g);
      float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
#pragma unroll
      for (int e = 0; e < PAIRS; ++e) {
        const float2 d = make_float2(g[2 * e], g[2 * e + 1]);  // (0 beyond the row)
        const float2 h = mul2(fma2(both(-mu[k]), one, make_float2(xh[2 * e], xh[2 * e + 1])), both(r[k]));
        dw[e] = fma2(d, h, dw[e]);
        db[e] = fma2(d, one, db[e]);
        s1 = fma2(d, w[e], s1);
        s2 = fma2(mul2(d, w[e]), h, s2);
      }
      s[2 * k] = s1.x + s1.y;
      s[2 * k + 1] = s2.x + s2.y;
    }
    if (dx) {
      float m1[2], m2[2];
      if constexpr (ROWS == 2) {
        const float4 m = row_sum4<TPR>(make_float4(s[0], s[1], s[2], s[3]), red, turn);
        m1[0] = m.x * inv;
        m2[0] = m.y * inv;
        m1[1] = m.z * inv;
        m2[1] = m.w * inv;
      } else {
        const float2 m = row_sum2<TPR>(s[0], s[1], reinterpret_cast<float2 *>(red), turn);
        m1[0] = m.x * inv;
        m2[0] = m.y * inv;
      }
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        if (row + k * step < a.rows) {
          float xh[EPT], g[EPT];
          if constexpr (ROWS == 2) take(k);  // (once more: kept over the barrier they spill)
          xb[k].get(xh);
          gb[k].get(g);
#pragma unroll
          for (int e = 0; e < PAIRS; ++e) {
            const float2 d = make_float2(g[2 * e], g[2 * e + 1]);
            const float2 h = mul2(fma2(both(-mu[k]), one, make_float2(xh[2 * e], xh[2 * e + 1])), both(r[k]));
            const float2 o = mul2(fma2(h, both(-m2[k]), fma2(d, w[e], both(-m1[k]))), both(r[k]));
            g[2 * e] = o.x;
            g[2 * e + 1] = o.y;
          }
          RowRegs<T, TPR, EPT, VEC>::store(dx + (row + k * step) * a.lddx, g, t, a.dim);
        }
        if constexpr (!RING) load(k, row + (k + ROWS) * step);
      }
    } else if constexpr (!RING) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k) load(k, row + (k + ROWS) * step);
    }
    if constexpr (RING) {
      fetch(stage, row + kNormStages * ROWS * step);  // (every word has been used)
      stage = stage + 1 < kNormStages ? stage + 1 : 0;
    }
  }
  if constexpr (RING) copy_wait_all();
  if (!a.partial) return;
  // One row of partial sums per row group: [2][gridDim.x * G][dim].
  float *pw = static_cast<float *>(a.partial);
  float *pb = pw + (long long)gridDim.x * G * a.dim;
  const long long at = ((long long)blockIdx.x * G + grp) * a.dim;
#pragma unroll
  for (int e = 0; e < EPT; ++e) {
    const int c = column<T, TPR, VEC>(t, e);
    if (c < a.dim) {
      pw[at + c] = e & 1 ? dw[e / 2].y : dw[e / 2].x;
      pb[at + c] = e & 1 ? db[e / 2].y : db[e / 2].x;
    }
  }
}

// Rows longer than a block's registers, and fp64: three walks over the row,
// the second and third of them in the caches.
template <typename T>
__global__ void __launch_bounds__(1024) layer_norm_long_kernel(const LayerNormArgs a) {
  using A = typename Acc<T>::type;
  __shared__ A red[2 * 32];
  int turn = 0;
  const A inv = (A)1 / (A)a.dim;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    T *y = static_cast<T *>(a.y) + row * a.ldy;
    A s = 0;
    for (int c = threadIdx.x; c < a.dim; c += 1024) s += to_acc(x[c]);
    const A mu = row_sum<1024>(s, red, turn) * inv;
    s = 0;
    for (int c = threadIdx.x; c < a.dim; c += 1024) {
      const A f = to_acc(x[c]) - mu;
      s += f * f;
    }
    const A r = (A)1 / sqrt(row_sum<1024>(s, red, turn) * inv + (A)a.eps);
    for (int c = threadIdx.x; c < a.dim; c += 1024) {
      A w = 1, b = 0;
      if constexpr (sizeof(T) == 8) {
        if (a.w) w = static_cast<const double *>(a.w)[c];
        if (a.b) b = static_cast<const double *>(a.b)[c];
      } else {
        if (a.w) w = load_any(a.w, a.wtype, c);
        if (a.b) b = load_any(a.b, a.wtype, c);
      }
      y[c] = from_acc<T>((to_acc(x[c]) - mu) * r * w + b);
    }
    if (threadIdx.x == 0) {
      if (a.mean) static_cast<A *>(a.mean)[row] = mu;
      if (a.rstd) static_cast<A *>(a.rstd)[row] = r;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(1024) layer_norm_long_dx_kernel(const LayerNormGradArgs a) {
  using A = typename Acc<T>::type;
  __shared__ A red[2 * 32];
  int turn = 0;
  const A inv = (A)1 / (A)a.dim;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    const T *dy = static_cast<const T *>(a.dy) + row * a.lddy;
    T *dx = static_cast<T *>(a.dx) + row * a.lddx;
    const A mu = static_cast<const A *>(a.mean)[row], r = static_cast<const A *>(a.rstd)[row];
    auto weight = [&](int c) -> A {
      if (!a.w) return 1;
      if constexpr (sizeof(T) == 8) return static_cast<const double *>(a.w)[c];
      else return load_any(a.w, a.wtype, c);
    };
    A s1 = 0, s2 = 0;
    for (int c = threadIdx.x; c < a.dim; c += 1024) {
      const A d = to_acc(dy[c]) * weight(c);
      s1 += d;
      s2 += d * (to_acc(x[c]) - mu) * r;
    }
    const A m1 = row_sum<1024>(s1, red, turn) * inv, m2 = row_sum<1024>(s2, red, turn) * inv;
    for (int c = threadIdx.x; c < a.dim; c += 1024) {
      const A xh = (to_acc(x[c]) - mu) * r;
      dx[c] = from_acc<T>(r * (to_acc(dy[c]) * weight(c) - m1 - xh * m2));
    }
  }
}

// Partial sums of dw and db over the rows blockIdx.y, + gridDim.y, ... of
// 256 columns.
template <typename T>
__global__ void __launch_bounds__(256) layer_norm_long_dw_kernel(const LayerNormGradArgs a) {
  using A = typename Acc<T>::type;
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.dim) return;
  const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);
  A dw = 0, db = 0;
  for (long long row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const A g = to_acc(dy[row * a.lddy + c]);
    dw += g * (to_acc(x[row * a.ldx + c]) - static_cast<const A *>(a.mean)[row]) *
          static_cast<const A *>(a.rstd)[row];
    db += g;
  }
  A *pw = static_cast<A *>(a.partial);
  pw[(long long)blockIdx.y * a.dim + c] = dw;
  pw[((long long)gridDim.y + blockIdx.y) * a.dim + c] = db;
}

// dw and db from `parts` rows of partial sums: 32 columns per block, 32
// threads down each column, added in a fixed order.  blockIdx.y: dw or db.
template <typename A>
__global__ void __launch_bounds__(1024)
layer_norm_sum_kernel(const A *partial, int parts, int dim, void *dw, void *db, int wtype) {
  __shared__ A tile[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  const A *p = partial + (long long)blockIdx.y * parts * dim;
  A s = 0;
  if (c < dim)
    for (int k = threadIdx.y; k < parts; k += 32) s += p[(long long)k * dim + c];
  tile[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = tile[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int col = blockIdx.x * 32 + threadIdx.y;
  void *out = blockIdx.y == 0 ? dw : db;
  if (threadIdx.x == 0 && col < dim && out) store_any(out, wtype, col, s);
}

// Threads per row and elements per thread by the row's length: a warp for rows
// up to 512 elements (no barrier), blocks of 128 to 1024 threads with 8
// elements each up to 8192; longer rows and fp64 by the looping kernels.  Few
// elements per thread leave room for many warps, which hide the barrier of a
// row's reduction (16 per thread, 256 threads: 90 us for 16384 x 4096 bf16
// forwards).  The gradients of that size take 83 us, 72% of the copy rate, and
// the sum of the partial rows 7: 16-bit rows are bound by their arithmetic (twice
// the elements per byte; fp32 rows reach 81%).  4096 bf16 rows of 8192 elements:
// 41 us forwards and 63 backwards, by the looping kernels 120 and 264.
constexpr int kNormRegMax = 8192;
inline int norm_tpr(int dim) {
  return dim <= 512 ? 32 : dim <= 1024 ? 128 : dim <= 2048 ? 256 : dim <= 4096 ? 512 : 1024;
}

template <typename T, class F>
cudaError_t norm_dispatch(int dim, bool vec, F f) {
#define FFTGB_NORM(TPR, EPT)                                      \
  return vec ? f(std::integral_constant<int, TPR>(), std::integral_constant<int, EPT>(), \
                 std::true_type())                                \
             : f(std::integral_constant<int, TPR>(), std::integral_constant<int, EPT>(), \
                 std::false_type())
  if (dim <= 256) { FFTGB_NORM(32, 8); }
  if (dim <= 512) { FFTGB_NORM(32, 16); }
  if (dim <= 1024) { FFTGB_NORM(128, 8); }
  if (dim <= 2048) { FFTGB_NORM(256, 8); }
  if (dim <= 4096) { FFTGB_NORM(512, 8); }
  FFTGB_NORM(1024, 8);
#undef FFTGB_NORM
}

inline int norm_groups(int dim) { return dim <= 512 ? 8 : 1; }  // row groups per block

// Blocks of the persistent kernels.
inline long long norm_grid(long long rows, int dim) {
  const int tpr = norm_tpr(dim);
  const long long blocks = (rows + norm_groups(dim) - 1) / norm_groups(dim);
  const long long most = (long long)sm_count() * (tpr == 32 ? 2 : tpr >= 1024 ? 1 : 1024 / tpr);
  return blocks < most ? blocks : most;
}

template <typename T> bool norm_vec(const void *p, long long ld, int dim) {
  return ((uintptr_t)p & 15u) == 0 && (ld * (long long)sizeof(T)) % 16 == 0 &&
         dim % Vec16<T>::N == 0;
}

template <typename T>
cudaError_t layer_norm_t(const LayerNormArgs &a, cudaStream_t st) {
  if constexpr (sizeof(T) < 8) {
    if (a.dim <= kNormRegMax) {
      const bool vec = norm_vec<T>(a.x, a.ldx, a.dim) && norm_vec<T>(a.y, a.ldy, a.dim);
      // Few long rows do not fill the multiprocessors with a warp or two each (bf16,
      // 152 SMs, us by warps and by blocks: 304 rows of 1024 2.9 and 2.4, of 2048 4.5
      // and 3.7, of 4096 5.0 and 5.5; 608 rows 3.3 and 3.4, 4.7 and 5.4, 5.6 and 7.2;
      // 1216 rows 4.0 and 5.3, 5.3 and 7.0, 7.7 and 10.3).
      if (vec && a.dim <= 16 * 32 * Vec16<T>::N && a.rows >= 4ll * sm_count())
        return layer_norm_warp<T>(a, st);
      const int grid = (int)norm_grid(a.rows, a.dim);
      return norm_dispatch<T>(a.dim, vec, [&](auto tpr, auto ept, auto v) {
        if constexpr (tpr.value == 32 && v.value) {
          return layer_norm_warp<T>(a, st);
        } else {
          layer_norm_kernel<T, tpr.value, ept.value, v.value>
              <<<grid, NormBlock<tpr.value>::THREADS, 0, st>>>(a);
          return cudaGetLastError();
        }
      });
    }
  }
  const long long most = 2LL * sm_count();
  layer_norm_long_kernel<T><<<(int)(a.rows < most ? a.rows : most), 1024, 0, st>>>(a);
  return cudaGetLastError();
}

// Row ranges of the looping kernel's dw: with 16, 64 and 256 of them the
// gradients of 512 bf16 rows of 12288 elements take 53, 56 and 66 us, of 64 rows
// 31, 32 and 30, of 4096 rows 373 each.
constexpr int kLongParts = 64;

template <typename T>
cudaError_t layer_norm_grad_t(const LayerNormGradArgs &a, cudaStream_t st) {
  using A = typename Acc<T>::type;
  const int dtype = sizeof(T) == 8 ? FFT_ELEM_F64 : FFT_ELEM_F32;
  const int parts = layer_norm_partials(dtype, a.rows, a.dim);
  cudaError_t e = cudaSuccess;
  bool done = false;
  if constexpr (sizeof(T) < 8) {
    if (a.dim <= kNormRegMax) {
      const bool vec = norm_vec<T>(a.x, a.ldx, a.dim) && norm_vec<T>(a.dy, a.lddy, a.dim) &&
                       (!a.dx || norm_vec<T>(a.dx, a.lddx, a.dim));
      const int grid = (int)norm_grid(a.rows, a.dim);
      e = norm_dispatch<T>(a.dim, vec, [&](auto tpr, auto ept, auto v) {
        constexpr size_t smem = norm_grad_smem<tpr.value, v.value>();
        auto kern = layer_norm_grad_kernel<T, tpr.value, ept.value, v.value>;
        if constexpr (smem > 0) {
          static DeviceOnce once;
          const cudaError_t limit = smem_limit_once((const void *)kern, smem, once);
          if (limit != cudaSuccess) return limit;
        }
        kern<<<grid, NormBlock<tpr.value>::THREADS, smem, st>>>(a);
        return cudaGetLastError();
      });
      done = true;
    }
  }
  if (!done) {
    // dw first: dx may overwrite dy or x.
    if (a.partial) {
      const dim3 grid((a.dim + 255) / 256, parts);
      layer_norm_long_dw_kernel<T><<<grid, 256, 0, st>>>(a);
      e = cudaGetLastError();
    }
    if (e == cudaSuccess && a.dx) {
      const long long most = 2LL * sm_count();
      layer_norm_long_dx_kernel<T><<<(int)(a.rows < most ? a.rows : most), 1024, 0, st>>>(a);
      e = cudaGetLastError();
    }
  }
  if (e == cudaSuccess && a.partial) {
    layer_norm_sum_kernel<A><<<dim3((a.dim + 31) / 32, 2), dim3(32, 32), 0, st>>>(
        static_cast<const A *>(a.partial), parts, a.dim, a.dw, a.db, a.wtype);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace fftgb
