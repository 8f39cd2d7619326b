// recur.cuh -- the gated linear recurrence, by channel,
//
//   h_t = a_t h_{t-1} + b_t x_t,  a_t = e^{g_t},  y_t = h_t,
//
// its gradients and single tokens.  With d_t the gradient of h_t and e_t that
// of h_{t-1} through token t, from the end
//
//   d_t = dy_t + e_{t+1},  e_t = a_t d_t,
//   dx_t = b_t d_t,  db_t = x_t d_t,  dg_t = e_t h_{t-1},  dh_0 = e_1.
//
// Both are bound by HBM if enough loads are under way.  A block of 8 warps has
// 128 channels, four per lane, and a warp 4 tokens of them at a time: its loads
// for the next step are issued before it waits for anything.  Tokens
// combine as maps h -> A h + H: each warp's into shared memory, each block's into
// the shared memory of the other blocks of a cluster, which has one sequence and
// walks it in steps of 32 tokens per block.  The state behind a step follows from the blocks'
// maps, which every block combines for itself, so a step has one barrier.
// Outputs are computed by the recurrence as it stands from the state in front of
// the warp's tokens: the maps only carry it there.
#pragma once

#include "cluster.cuh"
#include "seq.h"

namespace fftgb {
namespace {

constexpr int kRecurWarps = 8, kRecurTok = 4, kRecurWide = 128, kRecurBlocks = 8;

// Four channels of a lane as they are loaded: adjacent ones (VEC), or 32 apart.
template <typename T> struct Raw4 {
  T v[4];
};
template <typename T> struct alignas(4 * sizeof(T)) Vec4 {
  T v[4];
};
template <typename T, bool VEC> struct Lane4 {
  static __device__ __forceinline__ int at(int c0, int lane, int i) {
    return VEC ? c0 + 4 * lane + i : c0 + lane + 32 * i;
  }
  static __device__ __forceinline__ void load(Raw4<T> &r, const T *row, bool on, int c0, int lane,
                                              int channels) {
    if constexpr (VEC) {
      const int c = at(c0, lane, 0);
      Vec4<T> w{};
      if (on && c < channels) {
        if constexpr (sizeof(T) == 2) {
          const uint2 u = __ldg(reinterpret_cast<const uint2 *>(row + c));
          w = *reinterpret_cast<const Vec4<T> *>(&u);
        } else {
          const uint4 u = __ldg(reinterpret_cast<const uint4 *>(row + c));
          w = *reinterpret_cast<const Vec4<T> *>(&u);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) r.v[i] = w.v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = at(c0, lane, i);
        r.v[i] = on && c < channels ? __ldg(row + c) : from_acc<T>(0.0f);
      }
    }
  }
  static __device__ __forceinline__ void store(T *row, int c0, int lane, int channels,
                                               const float (&f)[4]) {
    if constexpr (VEC) {
      const int c = at(c0, lane, 0);
      if (c >= channels) return;
      Vec4<T> w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w.v[i] = from_acc<T>(f[i]);
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2 *>(row + c) = *reinterpret_cast<const uint2 *>(&w);
      else
        *reinterpret_cast<uint4 *>(row + c) = *reinterpret_cast<const uint4 *>(&w);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = at(c0, lane, i);
        if (c < channels) row[c] = from_acc<T>(f[i]);
      }
    }
  }
};

// A state of four channels, whose array needs no more than its elements' alignment
// (adjacent loads of a lane share their sectors).
template <bool VEC>
__device__ __forceinline__ void load_state(float (&f)[4], const float *row, int c0, int lane,
                                           int channels) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = Lane4<float, VEC>::at(c0, lane, i);
    f[i] = row && c < channels ? row[c] : 0.0f;
  }
}
template <bool VEC>
__device__ __forceinline__ void store_state(float *row, int c0, int lane, int channels,
                                            const float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = Lane4<float, VEC>::at(c0, lane, i);
    if (c < channels) row[c] = f[i];
  }
}

// A state behind a map.  A product of decays may be infinite where g > 0: it
// changes no state of 0.
__device__ __forceinline__ void apply(float4 A, float4 H, float (&s)[4]) {
  s[0] = s[0] == 0.0f ? H.x : fmaf(A.x, s[0], H.x);
  s[1] = s[1] == 0.0f ? H.y : fmaf(A.y, s[1], H.y);
  s[2] = s[2] == 0.0f ? H.z : fmaf(A.z, s[2], H.z);
  s[3] = s[3] == 0.0f ? H.w : fmaf(A.w, s[3], H.w);
}

struct RecurShared {
  float4 warp_a[2][kRecurWarps][32], warp_h[2][kRecurWarps][32];      // by step parity
  float4 block_a[2][kRecurBlocks][32], block_h[2][kRecurBlocks][32];  // of every block of the cluster
};

// Hands this warp's map round; afterwards s is the state in front of the warp's tokens
// and `carry` the one behind the whole step.
__device__ __forceinline__ void exchange(RecurShared &sh, int parity, int rank, int blocks,
                                         const float (&A)[4], const float (&H)[4],
                                         float (&carry)[4], float (&s)[4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  sh.warp_a[parity][warp][lane] = make_float4(A[0], A[1], A[2], A[3]);
  sh.warp_h[parity][warp][lane] = make_float4(H[0], H[1], H[2], H[3]);
  __syncthreads();
  if (blocks > 1) {
    if (warp < blocks) {  // warp w tells block w
      float4 a = sh.warp_a[parity][0][lane];
      const float4 h = sh.warp_h[parity][0][lane];
      float t[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
      for (int w = 1; w < kRecurWarps; ++w) {
        const float4 b = sh.warp_a[parity][w][lane];
        apply(b, sh.warp_h[parity][w][lane], t);
        a = make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
      }
      peer_store(peer((uint32_t)__cvta_generic_to_shared(&sh.block_a[parity][rank][lane]), warp), a);
      peer_store(peer((uint32_t)__cvta_generic_to_shared(&sh.block_h[parity][rank][lane]), warp),
                 make_float4(t[0], t[1], t[2], t[3]));
    }
    cluster_sync();
    for (int r = 0; r < blocks; ++r) {
      if (r == rank) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = carry[i];
      }
      apply(sh.block_a[parity][r][lane], sh.block_h[parity][r][lane], carry);
    }
#pragma unroll
    for (int w = 0; w < kRecurWarps - 1; ++w)
      if (w < warp) apply(sh.warp_a[parity][w][lane], sh.warp_h[parity][w][lane], s);
  } else {
#pragma unroll
    for (int w = 0; w < kRecurWarps; ++w) {
      if (w == warp) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = carry[i];
      }
      apply(sh.warp_a[parity][w][lane], sh.warp_h[parity][w][lane], carry);
    }
  }
}

// The rows of a sequence: offsets that descend or leave the rows are raised
// or cut to the nearest that do not.
struct Rows {
  long long begin, len;  // of the sequence
};
__device__ __forceinline__ Rows find_rows(const RecurArgs &a, long long seq) {
  __shared__ int found[2];
  Rows r;
  if (!a.offsets) {
    r.begin = seq * a.tokens;
    r.len = a.tokens;
    return r;
  }
  if (threadIdx.x < 2) found[threadIdx.x] = 0;
  __syncthreads();
  int m[2] = {0, 0};
  const int rows = (int)a.tokens;
  for (int i = threadIdx.x; i <= (int)seq + 1; i += blockDim.x) {
    const int v = min(max(a.offsets[i], 0), rows);
    if (i <= seq) m[0] = max(m[0], v);
    m[1] = max(m[1], v);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    m[k] = __reduce_max_sync(0xffffffffu, m[k]);
    if ((threadIdx.x & 31) == 0) atomicMax(&found[k], m[k]);
  }
  __syncthreads();
  r.begin = found[0];
  r.len = found[1] - found[0];
  return r;
}

// Rows of no sequence: before the first one's (its blocks) and behind the last one's.
template <typename T, bool VEC>
__device__ __forceinline__ void clear_rows(void *p, const RecurArgs &a, const Rows &r, long long seq,
                                           int rank, int c0) {
  if (!p) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float zero[4] = {0, 0, 0, 0};
  const int step = a.blocks * kRecurWarps, at = rank * kRecurWarps + warp;
  T *out = static_cast<T *>(p);
  if (seq == 0)
    for (long long t = at; t < r.begin; t += step)
      Lane4<T, VEC>::store(out + t * a.channels, c0, lane, a.channels, zero);
  if (seq == a.batch - 1)
    for (long long t = r.begin + r.len + at; t < a.tokens; t += step)
      Lane4<T, VEC>::store(out + t * a.channels, c0, lane, a.channels, zero);
}

// T: x and y; G: g and beta.
template <typename T, typename G, bool VEC, bool GATED>
__global__ void __launch_bounds__(kRecurWarps * 32, 2) recur_kernel(const RecurArgs a) {
  constexpr int K = kRecurTok;
  using LT = Lane4<T, VEC>;
  using LG = Lane4<G, VEC>;
  __shared__ RecurShared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = a.blocks > 1 ? (int)block_rank() : 0, C = a.channels;
  const long long unit = blockIdx.x / a.blocks;
  const int groups = (C + kRecurWide - 1) / kRecurWide;
  const long long seq = unit / groups;
  const int c0 = (int)(unit - seq * groups) * kRecurWide;
  const Rows r = find_rows(a, seq);
  if (a.clear) clear_rows<T, VEC>(a.y, a, r, seq, rank, c0);
  const long long from = a.offsets ? r.begin : 0, sq = a.offsets ? 0 : seq;
  const T *x = static_cast<const T *>(a.x) + sq * a.sx.seq + from * a.sx.tok;
  const G *g = static_cast<const G *>(a.g) + sq * a.sg.seq + from * a.sg.tok;
  const G *b = GATED ? static_cast<const G *>(a.beta) + sq * a.sb.seq + from * a.sb.tok : nullptr;
  T *y = static_cast<T *>(a.y) + r.begin * C;
  float carry[4];
  load_state<VEC>(carry, a.state_in ? a.state_in + seq * C : nullptr, c0, lane, C);
  if (a.blocks > 1) cluster_sync();  // every block's shared memory is there

  Raw4<T> rx[K];
  Raw4<G> rg[K], rb[K];
  auto fetch = [&](long long t0) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const long long t = t0 + j;
      const bool on = t < r.len;
      LT::load(rx[j], x + t * a.sx.tok, on, c0, lane, C);
      LG::load(rg[j], g + t * a.sg.tok, on, c0, lane, C);
      if constexpr (GATED) LG::load(rb[j], b + t * a.sb.tok, on, c0, lane, C);
    }
  };
  const int step = a.blocks * kRecurWarps * K;
  long long t0 = (long long)(rank * kRecurWarps + warp) * K;
  fetch(t0);
  int parity = 0;
  for (long long at = 0; at < r.len; at += step, t0 += step, parity ^= 1) {
    float e[K][4], u[K][4], A[4] = {1, 1, 1, 1}, H[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < K; ++j)  // behind the end g = x = 0: h stays
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e[j][i] = expf(to_acc(rg[j].v[i]));
        u[j][i] = to_acc(rx[j].v[i]);
        if constexpr (GATED) u[j][i] *= to_acc(rb[j].v[i]);
        A[i] *= e[j][i];
        H[i] = fmaf(e[j][i], H[i], u[j][i]);
      }
    fetch(t0 + step);
    float s[4];
    exchange(sh, parity, rank, a.blocks, A, H, carry, s);
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = fmaf(e[j][i], s[i], u[j][i]);
      if (t0 + j < r.len) LT::store(y + (t0 + j) * C, c0, lane, C, s);
    }
  }
  if (a.state_out && rank == 0 && warp == 0)
    store_state<VEC>(a.state_out + seq * C, c0, lane, C, carry);
}

// The same from the end: token len - 1 - t is the t-th.
template <typename T, typename G, bool VEC, bool GATED>
__global__ void __launch_bounds__(kRecurWarps * 32, 2) recur_grad_kernel(const RecurArgs a) {
  constexpr int K = kRecurTok;
  using LT = Lane4<T, VEC>;
  using LG = Lane4<G, VEC>;
  __shared__ RecurShared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = a.blocks > 1 ? (int)block_rank() : 0, C = a.channels;
  const long long unit = blockIdx.x / a.blocks;
  const int groups = (C + kRecurWide - 1) / kRecurWide;
  const long long seq = unit / groups;
  const int c0 = (int)(unit - seq * groups) * kRecurWide;
  const Rows r = find_rows(a, seq);
  if (a.clear) {
    clear_rows<T, VEC>(a.dx, a, r, seq, rank, c0);
    clear_rows<G, VEC>(a.dg, a, r, seq, rank, c0);
    if constexpr (GATED) clear_rows<G, VEC>(a.dbeta, a, r, seq, rank, c0);
  }
  const long long from = a.offsets ? r.begin : 0, sq = a.offsets ? 0 : seq;
  const T *x = static_cast<const T *>(a.x) + sq * a.sx.seq + from * a.sx.tok;
  const G *g = static_cast<const G *>(a.g) + sq * a.sg.seq + from * a.sg.tok;
  const G *b = GATED ? static_cast<const G *>(a.beta) + sq * a.sb.seq + from * a.sb.tok : nullptr;
  const T *y = static_cast<const T *>(a.y) + r.begin * C;
  const T *dy = static_cast<const T *>(a.dy) + r.begin * C;
  T *dx = static_cast<T *>(a.dx) + r.begin * C;
  G *dg = static_cast<G *>(a.dg) + r.begin * C;
  G *db = GATED ? static_cast<G *>(a.dbeta) + r.begin * C : nullptr;
  float carry[4];
  load_state<VEC>(carry, a.dfinal ? a.dfinal + seq * C : nullptr, c0, lane, C);
  if (a.blocks > 1) cluster_sync();

  Raw4<T> rd[K], ry[K], rx[K];
  Raw4<G> rg[K], rb[K];
  auto fetch = [&](long long t0) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const long long t = r.len - 1 - t0 - j;
      const bool on = t >= 0;
      LT::load(rd[j], dy + t * C, on, c0, lane, C);
      LG::load(rg[j], g + t * a.sg.tok, on, c0, lane, C);
      LT::load(ry[j], y + (t - 1) * C, t > 0, c0, lane, C);
      if constexpr (GATED) {
        LT::load(rx[j], x + t * a.sx.tok, on, c0, lane, C);
        LG::load(rb[j], b + t * a.sb.tok, on, c0, lane, C);
      }
    }
  };
  const int step = a.blocks * kRecurWarps * K;
  long long t0 = (long long)(rank * kRecurWarps + warp) * K;
  int parity = 0;
  fetch(t0);
  for (long long at = 0; at < r.len; at += step, t0 += step, parity ^= 1) {
    float e[K][4], d[K][4], A[4] = {1, 1, 1, 1}, H[4] = {0, 0, 0, 0};
    Raw4<T> ky[K], kx[K];
    Raw4<G> kb[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      ky[j] = ry[j];
      if constexpr (GATED) kx[j] = rx[j], kb[j] = rb[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e[j][i] = expf(to_acc(rg[j].v[i]));
        d[j][i] = to_acc(rd[j].v[i]);
        A[i] *= e[j][i];
        H[i] = e[j][i] * (H[i] + d[j][i]);
      }
    }
    fetch(t0 + step);
    float s[4];
    exchange(sh, parity, rank, a.blocks, A, H, carry, s);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const long long t = r.len - 1 - t0 - j;
      float before[4], o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) before[i] = to_acc(ky[j].v[i]);
      if (t == 0) load_state<VEC>(before, a.state_in ? a.state_in + seq * C : nullptr, c0, lane, C);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[j][i] += s[i];
        s[i] = e[j][i] * d[j][i];
      }
      if (t < 0) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = s[i] * before[i];
      LG::store(dg + t * C, c0, lane, C, o);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = GATED ? to_acc(kb[j].v[i]) * d[j][i] : d[j][i];
      LT::store(dx + t * C, c0, lane, C, o);
      if constexpr (GATED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = to_acc(kx[j].v[i]) * d[j][i];
        LG::store(db + t * C, c0, lane, C, o);
      }
    }
  }
  if (a.dinitial && rank == 0 && warp == 0)
    store_state<VEC>(a.dinitial + seq * C, c0, lane, C, carry);
}

// Single tokens: a thread has four channels of a sequence.
template <typename T, typename G, bool VEC, bool GATED>
__global__ void __launch_bounds__(128) recur_step_kernel(const RecurArgs a) {
  using LT = Lane4<T, VEC>;
  using LG = Lane4<G, VEC>;
  const int lane = threadIdx.x & 31, C = a.channels;
  const int groups = (C + kRecurWide - 1) / kRecurWide;
  const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const long long seq = unit / groups;
  if (seq >= a.batch) return;
  const int c0 = (int)(unit - seq * groups) * kRecurWide;
  const long long slot = a.slots ? a.slots[seq] : seq;
  const bool live = slot >= 0 && slot < a.pool;
  const T *x = static_cast<const T *>(a.x) + seq * a.sx.seq;
  const G *g = static_cast<const G *>(a.g) + seq * a.sg.seq;
  const G *b = GATED ? static_cast<const G *>(a.beta) + seq * a.sb.seq : nullptr;
  T *y = static_cast<T *>(a.y) + seq * a.tokens * C;
  float *state = live ? a.state_out + slot * C : nullptr;
  float h[4];
  load_state<VEC>(h, state, c0, lane, C);
  for (long long t = 0; t < a.tokens; ++t) {
    Raw4<T> rx;
    Raw4<G> rg, rb;
    LT::load(rx, x + t * a.sx.tok, live, c0, lane, C);
    LG::load(rg, g + t * a.sg.tok, live, c0, lane, C);
    if constexpr (GATED) LG::load(rb, b + t * a.sb.tok, live, c0, lane, C);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float u = to_acc(rx.v[i]);
      if constexpr (GATED) u *= to_acc(rb.v[i]);
      h[i] = fmaf(expf(to_acc(rg.v[i])), h[i], u);
    }
    LT::store(y + t * C, c0, lane, C, h);
  }
  if (live) store_state<VEC>(state, c0, lane, C, h);
}

// ---- launches ----------------------------------------------------------------------

// Rows of four channels that can be moved at once.
template <typename E> bool vec_rows4(const void *p, const RecurStride &s) {
  return ((uintptr_t)p & (4 * sizeof(E) - 1)) == 0 && s.seq % 4 == 0 && s.tok % 4 == 0;
}
template <typename T, typename G> bool vec_recur(const RecurArgs &a) {
  const RecurStride own{0, 0};
  return a.channels % 4 == 0 && vec_rows4<T>(a.x, a.sx) && vec_rows4<G>(a.g, a.sg) &&
         vec_rows4<G>(a.beta, a.sb) && vec_rows4<T>(a.y, own) && vec_rows4<T>(a.dy, own) &&
         vec_rows4<T>(a.dx, own) && vec_rows4<G>(a.dg, own) && vec_rows4<G>(a.dbeta, own);
}

template <typename F> cudaError_t launch_clusters(F *kern, RecurArgs a, cudaStream_t st) {
  const long long groups = (a.channels + kRecurWide - 1) / kRecurWide, units = a.batch * groups;
  const long long room = 2ll * sm_count();  // two blocks per SM
  if (room <= 0) return cudaErrorInvalidDevice;
  // Sequences share a GPU of many SMs: more blocks along one while there is
  // room for them and it has tokens for them.
  const long long mean = a.offsets ? (a.tokens + a.batch - 1) / a.batch : a.tokens;
  a.blocks = 1;
  while (a.blocks < kRecurBlocks && units * a.blocks * 2 <= room &&
         mean > (long long)a.blocks * kRecurWarps * kRecurTok)
    a.blocks *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(units * a.blocks));
  cfg.blockDim = dim3(kRecurWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)a.blocks;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.blocks > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, (const RecurArgs)a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, typename G, bool VEC, bool GATED>
cudaError_t recur_kind(int what, const RecurArgs &a, cudaStream_t st) {
  if (what == 0) return launch_clusters(&recur_kernel<T, G, VEC, GATED>, a, st);
  if (what == 1) return launch_clusters(&recur_grad_kernel<T, G, VEC, GATED>, a, st);
  const long long units = a.batch * ((a.channels + kRecurWide - 1) / kRecurWide);
  recur_step_kernel<T, G, VEC, GATED><<<(unsigned)((units + 3) / 4), 128, 0, st>>>(a);
  return cudaGetLastError();
}
template <typename T, typename G> cudaError_t recur_t(int what, const RecurArgs &a, cudaStream_t st) {
  if (vec_recur<T, G>(a))
    return a.beta ? recur_kind<T, G, true, true>(what, a, st)
                  : recur_kind<T, G, true, false>(what, a, st);
  return a.beta ? recur_kind<T, G, false, true>(what, a, st)
                : recur_kind<T, G, false, false>(what, a, st);
}
template <typename T> cudaError_t recur_of(int what, const RecurArgs &a, bool gfloat, cudaStream_t st) {
  if constexpr (sizeof(T) == 2)
    if (gfloat) return recur_t<T, float>(what, a, st);
  return recur_t<T, T>(what, a, st);
}

}  // namespace

template <typename T> cudaError_t launch_recur(const RecurArgs &a, bool gfloat, cudaStream_t st) {
  return recur_of<T>(0, a, gfloat, st);
}
template <typename T>
cudaError_t launch_recur_grad(const RecurArgs &a, bool gfloat, cudaStream_t st) {
  return recur_of<T>(1, a, gfloat, st);
}
template <typename T>
cudaError_t launch_recur_step(const RecurArgs &a, bool gfloat, cudaStream_t st) {
  return recur_of<T>(2, a, gfloat, st);
}

}  // namespace fftgb
