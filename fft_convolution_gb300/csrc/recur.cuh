// recur.cuh -- the gated linear recurrence, by channel,
//
//   h_t = a_t h_{t-1} + b_t x_t,  a_t = e^{g_t},  y_t = h_t,
//
// its gradients and single tokens.  With d_t the gradient of h_t and m_t that
// of h_{t-1} through token t, from the end
//
//   d_t = dy_t + m_{t+1},  m_t = a_t d_t,
//   dx_t = b_t d_t,  db_t = x_t d_t,  dg_t = m_t h_{t-1},  dh_0 = m_1.
//
// HBM is the bound, if enough loads are under way and little else is done: a
// block has 128 channels, four per lane of its 8 warps, and takes its tokens in
// tiles that the TMA brings two ahead.  A warp has K tokens of a tile.  Tokens
// combine as maps h -> A h + H: a warp's into shared memory, a block's (composed
// by all its warps, a few channels each) into the shared memory of the other
// blocks of its cluster, which share the sequence and walk it together, a tile
// each per step.  The maps carry the state to the front of each warp's tokens;
// outputs follow from there by the recurrence as it stands.
//
// Measured (bf16): 32768 tokens of 4096 channels 173 us, 8 x 4096 tokens of 2048
// channels backwards 176: 6.2 and 6.1 TB/s, 91% and 90% of a copy's rate.  In float
// 314 and 313, a copy's rate.
#pragma once

#include <cuda.h>

#include <stddef.h>

#include "cluster.cuh"
#include "seq.h"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace fftgb {
namespace {

constexpr int kRecurWarps = 8, kRecurThreads = 256, kRecurWide = 128, kRecurBlocks = 8, kRecurStages = 2;

// Four channels of a lane: adjacent ones (VEC: what the TMA brings as rows of 128
// channels), or 32 apart, which the lane's own copies put there.
template <typename T> struct alignas(4 * sizeof(T)) Four {
  T v[4];
};
template <typename T, bool VEC> struct Lane4 {
  static __device__ __forceinline__ int at(int c0, int lane, int i) {
    return VEC ? c0 + 4 * lane + i : c0 + lane + 32 * i;
  }
  // Copies them from a row to *dst: by asynchronous copies as far as there are
  // any of the elements' size.  Channels behind the last are left as they are.
  static __device__ __forceinline__ void fetch(Four<T> *dst, const T *row, int c0, int lane,
                                               int channels) {
    const uint32_t d = smem_u32(dst);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at(c0, lane, i) < channels)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d + 4 * i),
                       "l"(row + at(c0, lane, i))
                       : "memory");
    } else {
      Four<T> w;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w.v[i] = at(c0, lane, i) < channels ? __ldg(row + at(c0, lane, i)) : from_acc<T>(0.0f);
      *dst = w;
    }
  }
  static __device__ __forceinline__ void store(T *row, int c0, int lane, int channels,
                                               const float (&f)[4]) {
    if constexpr (VEC) {
      const int c = at(c0, lane, 0);
      if (c >= channels) return;
      Four<T> w;
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
  // Straight from global memory.
  static __device__ __forceinline__ void load(float (&f)[4], const T *row, bool on, int c0, int lane,
                                              int channels) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = at(c0, lane, i);
      f[i] = on && c < channels ? to_acc(row[c]) : 0.0f;
    }
  }
};
// Four channels as two pairs, which most instructions take at once.
struct Pairs {
  float2 p[2];
};
__device__ __forceinline__ Pairs widen(const Four<float> &v) {
  return Pairs{{make_float2(v.v[0], v.v[1]), make_float2(v.v[2], v.v[3])}};
}
__device__ __forceinline__ Pairs widen(const Four<__half> &v) {
  const uint2 u = *reinterpret_cast<const uint2 *>(&v);
  return Pairs{{__half22float2(*reinterpret_cast<const __half2 *>(&u.x)),
                __half22float2(*reinterpret_cast<const __half2 *>(&u.y))}};
}
__device__ __forceinline__ Pairs widen(const Four<__nv_bfloat16> &v) {
  const uint2 u = *reinterpret_cast<const uint2 *>(&v);
  return Pairs{{make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u)),
                make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u))}};
}
__device__ __forceinline__ Pairs operator*(const Pairs &a, const Pairs &b) {
  return Pairs{{mul2(a.p[0], b.p[0]), mul2(a.p[1], b.p[1])}};
}
__device__ __forceinline__ Pairs fma4(const Pairs &a, const Pairs &b, const Pairs &c) {
  return Pairs{{fma2(a.p[0], b.p[0], c.p[0]), fma2(a.p[1], b.p[1], c.p[1])}};
}
__device__ __forceinline__ Pairs splat(float v) { return Pairs{{both(v), both(v)}}; }
// e^g as 2^(g log2 e): off by about 2^-23, and by |g| 2^-24 more through the product's
// rounding.
__device__ __forceinline__ Pairs decay(const Pairs &g) {
  Pairs t = g * splat(1.4426950408889634f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t.p[i].x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t.p[i].y));
  }
  return t;
}
__device__ __forceinline__ void unpair(const Pairs &a, float (&f)[4]) {
  f[0] = a.p[0].x;
  f[1] = a.p[0].y;
  f[2] = a.p[1].x;
  f[3] = a.p[1].y;
}
__device__ __forceinline__ Pairs pair_up(const float (&f)[4]) {
  return Pairs{{make_float2(f[0], f[1]), make_float2(f[2], f[3])}};
}
__device__ __forceinline__ Pairs pair_up(float4 v) {
  return Pairs{{make_float2(v.x, v.y), make_float2(v.z, v.w)}};
}
__device__ __forceinline__ float4 quad(const Pairs &a) {
  return make_float4(a.p[0].x, a.p[0].y, a.p[1].x, a.p[1].y);
}
// A product of decays (all of them finite and none below 0), taken without bounds, as maps
// hand it on. Above float's range (g > 0) it ends at the largest value, which leaves a
// state of 0 alone where infinity would not. Infinity stays infinity under every factor
// but 0, which makes it NaN for good: then the product has a factor of 0 and is 0. (A g
// that is NaN or infinite shows in the map's other half.) A bound at every factor would
// take 178.7 us instead of 171.7 for 32768 tokens of 4096 channels.
__device__ __forceinline__ Pairs bounded(Pairs a) {
  constexpr float most = 3.402823466e38f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    a.p[i].x = fminf(fmaxf(a.p[i].x, 0.0f), most);  // fmaxf(NaN, 0) is 0
    a.p[i].y = fminf(fmaxf(a.p[i].y, 0.0f), most);
  }
  return a;
}

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

struct RecurShared {
  // maps h -> a h + h0 of the warps, of the cluster's blocks by step parity, and the
  // states in front of the warps' tokens: of four channels each
  float4 warp_a[kRecurWarps][32], warp_h[kRecurWarps][32];
  float4 block_a[2][kRecurBlocks][32], block_h[2][kRecurBlocks][32];
  float4 state[kRecurWarps][32];
  uint64_t full[kRecurStages];  // the stages' tiles have come
  uint64_t sent[2];  // the blocks' maps have come
  // A wait has run out: for a tile, for maps.  All threads look at each behind a
  // barrier that everyone who may set it has passed, so they leave together.
  int failed[2];
};
constexpr size_t kRecurShared = (sizeof(RecurShared) + 127) / 128 * 128;
// Behind it the stages: of each input a tile of tokens x 128 channels.

__device__ __forceinline__ void exchange_begin(RecurShared &sh, const Waits &waits) {
  if (threadIdx.x == 0) {
    const int starved = blockIdx.x == 0 ? waits.starved : 0;  // one arrival more than will come
    for (int i = 0; i < kRecurStages; ++i) bar_init(&sh.full[i], starved == 1 + i ? 2 : 1);
    for (int i = 0; i < 2; ++i) bar_init(&sh.sent[i], starved == 3 + i ? 2 : 1);
    sh.failed[0] = sh.failed[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
}

// Every block's shared memory is there, and what it reads of the first state has been read:
// the last state, which one of them writes, may lie in the same place.
__device__ __forceinline__ void exchange_ready(int blocks) {
  __syncwarp();
  if (blocks > 1) cluster_sync();
}

// No block leaves before the others have sent their last map, and none that has given up before
// those have come.
__device__ __forceinline__ void exchange_end(const RecurShared &sh, int blocks) {
  __syncwarp();
  if (blocks == 1) return;
  cluster_sync();
  if (sh.failed[0] | sh.failed[1]) linger();
}

// A lane's share of an exchange: channels 4 quad .. of the tile, for the block
// (then the warp) `to`.  Eight lanes have the same channels: their loads are one.
struct Share {
  int quad, to;
};
__device__ __forceinline__ Share my_share() {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  return Share{4 * warp + (lane & 3), lane >> 2};
}

// Step n, all of a block's warps: hands the warp's map A h + H round, after
// which s is the state in front of the warp's tokens, and `carry` (of the lane's share)
// the one behind the step.  `between` runs when every warp has come here.
// False: a wait has run out.
// A block map's buffer is written again two steps later: by a block that has the
// maps of the step between, which are sent when all warps have read the older ones.
template <class Between>
__device__ __forceinline__ bool exchange(RecurShared &sh, uint32_t n, int rank, int blocks,
                                         const Pairs &A, const Pairs &H, Pairs &carry, Pairs &s,
                                         int *status, long long limit, Between between) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, parity = n & 1;
  const Share my = my_share();
  sh.warp_a[warp][lane] = quad(bounded(A));
  sh.warp_h[warp][lane] = quad(H);
  __syncthreads();
  if (*(volatile int *)&sh.failed[0]) return false;
  between();
  Pairs a[kRecurWarps], h[kRecurWarps];
#pragma unroll
  for (int w = 0; w < kRecurWarps; ++w) {
    a[w] = pair_up(sh.warp_a[w][my.quad]);
    h[w] = pair_up(sh.warp_h[w][my.quad]);
  }
  if (blocks > 1) {
    if (threadIdx.x == 0) bar_arrive_tx(&sh.sent[parity], (uint32_t)blocks * 1024);
    Pairs all_a = a[0], all_h = h[0];
#pragma unroll
    for (int w = 1; w < kRecurWarps; ++w) {
      all_h = fma4(a[w], all_h, h[w]);
      all_a = all_a * a[w];
    }
    if (my.to < blocks) {
      const uint32_t bar = peer(smem_u32(&sh.sent[parity]), my.to);
      peer_send(peer(smem_u32(&sh.block_a[parity][rank][my.quad]), my.to), quad(bounded(all_a)), bar);
      peer_send(peer(smem_u32(&sh.block_h[parity][rank][my.quad]), my.to), quad(all_h), bar);
    }
    wait_cluster(&sh.sent[parity], (n >> 1) & 1, &sh.failed[1], status, limit);
    s = carry;
#pragma unroll
    for (int r = 0; r < kRecurBlocks; ++r)
      if (r < blocks) {
        if (r == rank) s = carry;
        carry = fma4(pair_up(sh.block_a[parity][r][my.quad]), carry,
                     pair_up(sh.block_h[parity][r][my.quad]));
      }
  } else {
    s = carry;
#pragma unroll
    for (int w = 0; w < kRecurWarps; ++w) carry = fma4(a[w], carry, h[w]);
  }
#pragma unroll
  for (int w = 0; w < kRecurWarps - 1; ++w)
    if (w < my.to) s = fma4(a[w], s, h[w]);
  sh.state[my.to][my.quad] = quad(s);
  __syncthreads();
  s = pair_up(sh.state[warp][lane]);
  return *(volatile int *)&sh.failed[1] == 0;
}

// A tile of `rows` tokens of 128 channels, counted by the barrier.
__device__ __forceinline__ void tile_load(void *dst, const CUtensorMap *map, int c, int t, int seq,
                                          uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c), "r"(t), "r"(seq)
      : "memory");
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
  if (a.rows) {
    r.begin = a.rows[seq];
    r.len = a.rows[seq + 1] - r.begin;
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

// The inputs' tensor maps, where the TMA loads them (VEC): x, g, beta, dy, y.
struct RecurMaps {
  CUtensorMap x, g, b, d, y;
};
// Tokens of a warp per step, where a lane's loads of one take `bytes`: two stages
// of tiles fill shared memory, one block per SM.  A step costs about 1500 clocks
// beside its tokens, so many small ones lose (prompt of 32768 tokens, 4096
// channels in bf16: 170 us with 16 tokens, 252 with 8, 301 with 4).  SHORT sequences
// are all start and end: small tiles, two blocks per SM (4096 sequences of 16 tokens,
// 1024 channels: 743 -> 273 us, 512 of 64 107 -> 63, 256 of 128 65 -> 57, but 64 of
// 1024 92 -> 104). Of packed sequences it is the mean length that decides, as the host
// does not know the offsets: one long among many short ones loses (16000 tokens and 500
// times 16, 1024 channels: 537 us in small tiles, 281 in large ones).
constexpr int kRecurShort = 192;
constexpr int recur_tokens(int bytes, bool is_short) {
  return is_short ? (bytes <= 40 ? 4 : 2) : bytes <= 24 ? 16 : bytes <= 48 ? 8 : 4;
}

// T: x and y; G: g and beta.
template <typename T, typename G, bool GATED, bool SHORT> struct RecurForward {
  static constexpr int K = recur_tokens(4 * (int)(sizeof(T) + sizeof(G) * (GATED ? 2 : 1)), SHORT);
  static constexpr int kTokens = kRecurWarps * K, S = kRecurStages;
  struct Stage {
    alignas(128) Four<T> x[kTokens][32];
    alignas(128) Four<G> g[kTokens][32];
    alignas(128) Four<G> b[GATED ? kTokens : 1][GATED ? 32 : 1];
  };
  static_assert(sizeof(Stage) % 128 == 0 && offsetof(Stage, g) % 128 == 0 && offsetof(Stage, b) % 128 == 0, "TMA");
  static constexpr uint32_t kBytes = kTokens * 128 * (sizeof(T) + sizeof(G) * (GATED ? 2 : 1));
  static constexpr size_t kSmem = 128 + kRecurShared + S * sizeof(Stage);
};
template <typename T, typename G, bool VEC, bool GATED, bool SHORT>
__global__ void __launch_bounds__(kRecurThreads, SHORT ? 2 : 1)
recur_kernel(const RecurArgs a, const __grid_constant__ RecurMaps maps, int *status) {
  using P = RecurForward<T, G, GATED, SHORT>;
  constexpr int K = P::K, S = P::S;
  using LT = Lane4<T, VEC>;
  using LG = Lane4<G, VEC>;
  extern __shared__ char smem_raw[];
  char *smem = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
  RecurShared &sh = *reinterpret_cast<RecurShared *>(smem);
  auto stage = [&](uint32_t n) -> typename P::Stage & {
    return *reinterpret_cast<typename P::Stage *>(smem + kRecurShared +
                                                  (n % S) * sizeof(typename P::Stage));
  };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  const int step = a.blocks * P::kTokens;
  exchange_begin(sh, a.waits);

  // The tile of step n, from its first token on: the TMA for the whole block
  // (thread 0), or this lane's part of it.
  auto fetch = [&](uint32_t n) {
    const long long t0 = (long long)n * step + rank * P::kTokens;
    typename P::Stage &st = stage(n);
    if constexpr (VEC) {
      if (tid != 0 || t0 >= r.len) return;
      const int t = (int)(from + t0);
      bar_arrive_tx(&sh.full[n % S], P::kBytes);
      tile_load(&st.x, &maps.x, c0, t, (int)sq, &sh.full[n % S]);
      tile_load(&st.g, &maps.g, c0, t, (int)sq, &sh.full[n % S]);
      if constexpr (GATED) tile_load(&st.b, &maps.b, c0, t, (int)sq, &sh.full[n % S]);
    } else {
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const long long t = t0 + warp * K + j;
        if (t < r.len) {
          LT::fetch(&st.x[warp * K + j][lane], x + t * a.sx.tok, c0, lane, C);
          LG::fetch(&st.g[warp * K + j][lane], g + t * a.sg.tok, c0, lane, C);
          if constexpr (GATED) LG::fetch(&st.b[warp * K + j][lane], b + t * a.sb.tok, c0, lane, C);
        }
      }
      copy_group();
    }
  };
  for (uint32_t n = 0; n < S; ++n) fetch(n);
  float state[4];
  const Share my = my_share();
  load_state<VEC>(state, a.state_in ? a.state_in + seq * C : nullptr, c0, my.quad, C);
  Pairs carry = pair_up(state);
  exchange_ready(a.blocks);
  uint32_t n = 0;
  for (long long at = 0; at < r.len; at += step, ++n) {
    const long long t0 = at + rank * P::kTokens + warp * K;
    const int count = (int)max(0ll, min((long long)K, r.len - t0));
    Pairs e[K], u[K], A = splat(1.0f), H = splat(0.0f), h;
    if constexpr (VEC) {
      if (at + rank * P::kTokens < r.len)
        wait_cluster(&sh.full[n % S], (n / S) & 1, &sh.failed[0], status, a.waits.limit);
    } else {
      copy_wait<S - 1>();
    }
    const typename P::Stage &st = stage(n);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (j < count) {
        e[j] = decay(widen(st.g[warp * K + j][lane]));
        u[j] = widen(st.x[warp * K + j][lane]);
        if constexpr (GATED) u[j] = u[j] * widen(st.b[warp * K + j][lane]);
        A = A * e[j];
        H = fma4(e[j], H, u[j]);
      }
    }
    if constexpr (!VEC) fetch(n + S);
    if (!exchange(sh, n, rank, a.blocks, A, H, carry, h, status, a.waits.limit, [&] {
          if constexpr (VEC) fetch(n + S);  // every warp has read the tile
        }))
      break;
    T *py = y + t0 * C;
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (j < count) {
        h = fma4(e[j], h, u[j]);
        float o[4];
        unpair(h, o);
        LT::store(py, c0, lane, C, o);
        py += C;
      }
  }
  if (a.state_out && rank == 0 && my.to == 0) {
    unpair(carry, state);
    store_state<VEC>(a.state_out + seq * C, c0, my.quad, C, state);
  }
  // Given up: no copy may land after the block has gone. Tiles n .. n + S - 1 have been asked
  // for, and the one behind them where the step came as far as the blocks' maps.
  if (sh.failed[0] | sh.failed[1]) {
    if constexpr (VEC) {
      const uint32_t end = n + S + (sh.failed[1] ? 1 : 0);
#pragma unroll 1
      for (uint32_t i = n; tid == 0 && i < end; ++i)
        if ((long long)i * step + rank * P::kTokens < r.len) let_land(&sh.full[i % S], (i / S) & 1);
    } else {
      copy_wait_all();
    }
  }
  exchange_end(sh, a.blocks);
}

// The same from the end: tile n has the tokens behind those of tile n + 1, and a
// warp's j-th token is the j-th from its end.
template <typename T, typename G, bool GATED, bool SHORT> struct RecurBackward {
  // more than 8 would not leave registers for both factors of a token
  static constexpr int kMost =
      recur_tokens(4 * (int)(sizeof(T) * (GATED ? 3 : 2) + sizeof(G) * (GATED ? 2 : 1)), SHORT);
  static constexpr int K = kMost < 8 ? kMost : 8;
  static constexpr int kTokens = kRecurWarps * K, S = kRecurStages;
  struct Stage {
    alignas(128) Four<T> d[kTokens][32];
    alignas(128) Four<T> y[kTokens][32];
    alignas(128) Four<G> g[kTokens][32];
    alignas(128) Four<T> x[GATED ? kTokens : 1][GATED ? 32 : 1];
    alignas(128) Four<G> b[GATED ? kTokens : 1][GATED ? 32 : 1];
  };
  static_assert(sizeof(Stage) % 128 == 0 && offsetof(Stage, y) % 128 == 0 && offsetof(Stage, g) % 128 == 0 &&
                    offsetof(Stage, x) % 128 == 0 && offsetof(Stage, b) % 128 == 0,
                "TMA");
  static constexpr uint32_t kBytes =
      kTokens * 128 * (sizeof(T) * (GATED ? 3 : 2) + sizeof(G) * (GATED ? 2 : 1));
  static constexpr size_t kSmem = 128 + kRecurShared + S * sizeof(Stage);
};
template <typename T, typename G, bool VEC, bool GATED, bool SHORT>
__global__ void __launch_bounds__(kRecurThreads, SHORT ? 2 : 1)
recur_grad_kernel(const RecurArgs a, const __grid_constant__ RecurMaps maps, int *status) {
  using P = RecurBackward<T, G, GATED, SHORT>;
  constexpr int K = P::K, S = P::S;
  using LT = Lane4<T, VEC>;
  using LG = Lane4<G, VEC>;
  extern __shared__ char smem_raw[];
  char *smem = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
  RecurShared &sh = *reinterpret_cast<RecurShared *>(smem);
  auto stage = [&](uint32_t n) -> typename P::Stage & {
    return *reinterpret_cast<typename P::Stage *>(smem + kRecurShared +
                                                  (n % S) * sizeof(typename P::Stage));
  };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  const int step = a.blocks * P::kTokens;
  exchange_begin(sh, a.waits);

  auto fetch = [&](uint32_t n) {
    const long long last = r.len - 1 - ((long long)n * step + rank * P::kTokens);  // its last token
    typename P::Stage &st = stage(n);
    if constexpr (VEC) {
      if (tid != 0 || last < 0) return;
      const int t = (int)(from + last) - (P::kTokens - 1);
      uint64_t *bar = &sh.full[n % S];
      bar_arrive_tx(bar, P::kBytes);
      tile_load(&st.d, &maps.d, c0, t, (int)sq, bar);
      tile_load(&st.g, &maps.g, c0, t, (int)sq, bar);
      tile_load(&st.y, &maps.y, c0, t - 1, (int)sq, bar);
      if constexpr (GATED) {
        tile_load(&st.x, &maps.x, c0, t, (int)sq, bar);
        tile_load(&st.b, &maps.b, c0, t, (int)sq, bar);
      }
    } else {
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const long long t = last - warp * K - j;
        const int row = P::kTokens - 1 - warp * K - j;
        if (t >= 0) {
          LT::fetch(&st.d[row][lane], dy + t * C, c0, lane, C);
          LG::fetch(&st.g[row][lane], g + t * a.sg.tok, c0, lane, C);
          if (t > 0) LT::fetch(&st.y[row][lane], y + (t - 1) * C, c0, lane, C);
          if constexpr (GATED) {
            LT::fetch(&st.x[row][lane], x + t * a.sx.tok, c0, lane, C);
            LG::fetch(&st.b[row][lane], b + t * a.sb.tok, c0, lane, C);
          }
        }
      }
      copy_group();
    }
  };
  for (uint32_t n = 0; n < S; ++n) fetch(n);
  float state[4];
  const Share my = my_share();
  load_state<VEC>(state, a.dfinal ? a.dfinal + seq * C : nullptr, c0, my.quad, C);
  Pairs carry = pair_up(state);
  exchange_ready(a.blocks);
  uint32_t n = 0;
  for (long long at = 0; at < r.len; at += step, ++n) {
    const long long t0 = r.len - 1 - at - rank * P::kTokens - warp * K;
    const int count = (int)max(0ll, min((long long)K, t0 + 1));
    const int row = P::kTokens - 1 - warp * K;
    Pairs e[K], d[K], A = splat(1.0f), H = splat(0.0f), m;
    if constexpr (VEC) {
      if (at + rank * P::kTokens < r.len)
        wait_cluster(&sh.full[n % S], (n / S) & 1, &sh.failed[0], status, a.waits.limit);
    } else {
      copy_wait<S - 1>();
    }
    const typename P::Stage &st = stage(n);
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (j < count) {
        e[j] = decay(widen(st.g[row - j][lane]));
        d[j] = widen(st.d[row - j][lane]);
        A = A * e[j];
        H = fma4(e[j], H, e[j] * d[j]);
      }
    if (!exchange(sh, n, rank, a.blocks, A, H, carry, m, status, a.waits.limit, [&] {
          // every warp is done with the tile before this one
          if (VEC && n > 0) fetch(n - 1 + S);
        }))
      break;
    T *px = dx + t0 * C;
    G *pg = dg + t0 * C, *pb = GATED ? db + t0 * C : nullptr;
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (j < count) {
        const Pairs now = Pairs{{make_float2(m.p[0].x + d[j].p[0].x, m.p[0].y + d[j].p[0].y),
                                 make_float2(m.p[1].x + d[j].p[1].x, m.p[1].y + d[j].p[1].y)}};
        m = e[j] * now;
        Pairs before = widen(st.y[row - j][lane]);
        if (j == t0) {
          load_state<VEC>(state, a.state_in ? a.state_in + seq * C : nullptr, c0, lane, C);
          before = pair_up(state);
        }
        float o[4];
        unpair(m * before, o);
        LG::store(pg, c0, lane, C, o);
        Pairs out = now;
        if constexpr (GATED) {
          unpair(now * widen(st.x[row - j][lane]), o);
          LG::store(pb, c0, lane, C, o);
          out = now * widen(st.b[row - j][lane]);
        }
        unpair(out, o);
        LT::store(px, c0, lane, C, o);
        px -= C;
        pg -= C;
        if constexpr (GATED) pb -= C;
      }
    if constexpr (!VEC) fetch(n + S);
  }
  if (a.dinitial && rank == 0 && my.to == 0) {
    unpair(carry, state);
    store_state<VEC>(a.dinitial + seq * C, c0, my.quad, C, state);
  }
  // Given up, as forward: tile n - 1 + S has been asked for in step n, as far as that came.
  if (sh.failed[0] | sh.failed[1]) {
    if constexpr (VEC) {
      const uint32_t end = n + S - (sh.failed[0] && n > 0 ? 1 : 0);
#pragma unroll 1
      for (uint32_t i = n; tid == 0 && i < end; ++i)
        if ((long long)i * step + rank * P::kTokens < r.len) let_land(&sh.full[i % S], (i / S) & 1);
    } else {
      copy_wait_all();
    }
  }
  exchange_end(sh, a.blocks);
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
    float fx[4], fg[4], fb[4];
    LT::load(fx, x + t * a.sx.tok, live, c0, lane, C);
    LG::load(fg, g + t * a.sg.tok, live, c0, lane, C);
    if constexpr (GATED) LG::load(fb, b + t * a.sb.tok, live, c0, lane, C);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (GATED) fx[i] *= fb[i];
      h[i] = fmaf(expf(fg[i]), h[i], fx[i]);
    }
    LT::store(y + t * C, c0, lane, C, h);
  }
  if (live) store_state<VEC>(state, c0, lane, C, h);
}

// ---- launches ----------------------------------------------------------------------

// The map of an array [sequence][token][channel] (packed: [1][row][channel])
// in tiles of `tokens` x 128 channels; false where the TMA cannot take its rows.
template <typename E>
bool recur_map(CUtensorMap *map, const void *p, const RecurStride &s, const RecurArgs &a, int tokens) {
  const long long seqs = a.offsets ? 1 : a.batch, bytes = (long long)sizeof(E);
  const long long tok = a.tokens > 1 ? s.tok * bytes : 16;
  const long long seq = seqs > 1 ? s.seq * bytes : tok;
  const TensorMapEncodeFn fn = tensor_map_encode();
  if (!fn || ((uintptr_t)p & 15) != 0 || a.channels % 4 != 0 || tok <= 0 || seq <= 0 || tok % 16 != 0 ||
      seq % 16 != 0 || tok >= (1ll << 40) || seq >= (1ll << 40) || a.tokens == 0)
    return false;
  const cuuint64_t dims[3] = {(cuuint64_t)a.channels, (cuuint64_t)a.tokens, (cuuint64_t)seqs};
  const cuuint64_t strides[2] = {(cuuint64_t)tok, (cuuint64_t)seq};
  const cuuint32_t box[3] = {kRecurWide, (cuuint32_t)tokens, 1}, ones[3] = {1, 1, 1};
  const CUtensorMapDataType type = sizeof(E) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                  : CU_TENSOR_MAP_DATA_TYPE_UINT16;
  return fn(map, type, 3, const_cast<void *>(p), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Outputs in stores of four elements.
template <typename E> bool quads(const void *p) { return ((uintptr_t)p & (4 * sizeof(E) - 1)) == 0; }

template <typename F>
cudaError_t launch_clusters(F *kern, RecurArgs a, const RecurMaps &maps, int tokens, size_t smem,
                            DeviceOnce &once, std::atomic<int> (&resident)[64], cudaStream_t st) {
  int *status = device_status_word();
  if (!status) return cudaErrorInvalidDevice;
  cudaError_t e = smem_limit_once((const void *)kern, smem, once);
  if (e != cudaSuccess) return e;
  const long long groups = (a.channels + kRecurWide - 1) / kRecurWide, units = a.batch * groups;
  const long long room =
      (long long)sm_count() * blocks_per_sm_once((const void *)kern, kRecurThreads, smem, resident);
  if (room <= 0) return cudaErrorInvalidDevice;
  if (a.rows) {  // a block would read all offsets before its own
    e = launch_delta_plan(a.offsets, a.batch, a.tokens, a.rows, a.rows + a.batch + 1, DeltaClear{}, st);
    if (e != cudaSuccess) return e;
  }
  // Sequences share a GPU of many SMs: more blocks along one while there is
  // room for them and it has tokens for them.
  const long long mean = a.offsets ? (a.tokens + a.batch - 1) / a.batch : a.tokens;
  a.waits = waits_now();
  a.blocks = 1;
  while (a.blocks < kRecurBlocks && units * a.blocks * 2 <= room &&
         mean > (long long)a.blocks * tokens)
    a.blocks *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(units * a.blocks));
  cfg.blockDim = dim3(kRecurThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)a.blocks;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.blocks > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, (const RecurArgs)a, maps, status);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, typename G, bool GATED, bool SHORT>
cudaError_t recur_whole(bool grad, const RecurArgs &a, cudaStream_t st) {
  using F = RecurForward<T, G, GATED, SHORT>;
  using B = RecurBackward<T, G, GATED, SHORT>;
  RecurMaps maps{};
  const RecurStride own{a.tokens * a.channels, a.channels};
  const int tokens = grad ? B::kTokens : F::kTokens;
  const size_t smem = grad ? B::kSmem : F::kSmem;
  bool vec = quads<T>(a.y) && recur_map<G>(&maps.g, a.g, a.sg, a, tokens);
  if (GATED) vec = vec && recur_map<G>(&maps.b, a.beta, a.sb, a, tokens);
  if (GATED || !grad) vec = vec && recur_map<T>(&maps.x, a.x, a.sx, a, tokens);
  if (grad)
    vec = vec && quads<T>(a.dx) && quads<G>(a.dg) && quads<G>(a.dbeta) &&
          recur_map<T>(&maps.d, a.dy, own, a, tokens) && recur_map<T>(&maps.y, a.y, own, a, tokens);
  static DeviceOnce once[4];
  static std::atomic<int> resident[4][64];
  auto kern = grad ? (vec ? &recur_grad_kernel<T, G, true, GATED, SHORT>
                          : &recur_grad_kernel<T, G, false, GATED, SHORT>)
                   : (vec ? &recur_kernel<T, G, true, GATED, SHORT>
                          : &recur_kernel<T, G, false, GATED, SHORT>);
  const int which = (grad ? 2 : 0) + (vec ? 1 : 0);
  return launch_clusters(kern, a, maps, tokens, smem, once[which], resident[which], st);
}
template <typename T, typename G, bool GATED>
cudaError_t recur_kind(int what, const RecurArgs &a, cudaStream_t st) {
  if (what == 2) {
    const auto fits = [&](const void *p, const RecurStride &s, size_t e) {
      return ((uintptr_t)p & (4 * e - 1)) == 0 && s.seq % 4 == 0 && s.tok % 4 == 0;
    };
    const bool vec = a.channels % 4 == 0 && quads<T>(a.y) && fits(a.x, a.sx, sizeof(T)) &&
                     fits(a.g, a.sg, sizeof(G)) && fits(a.beta, a.sb, sizeof(G));
    const long long units = a.batch * ((a.channels + kRecurWide - 1) / kRecurWide);
    const unsigned grid = (unsigned)((units + 3) / 4);
    if (vec) recur_step_kernel<T, G, true, GATED><<<grid, 128, 0, st>>>(a);
    else recur_step_kernel<T, G, false, GATED><<<grid, 128, 0, st>>>(a);
    return cudaGetLastError();
  }
  const long long mean = a.offsets ? a.tokens / a.batch : a.tokens;
  return mean <= kRecurShort ? recur_whole<T, G, GATED, true>(what == 1, a, st)
                             : recur_whole<T, G, GATED, false>(what == 1, a, st);
}
template <typename T, typename G> cudaError_t recur_t(int what, const RecurArgs &a, cudaStream_t st) {
  return a.beta ? recur_kind<T, G, true>(what, a, st) : recur_kind<T, G, false>(what, a, st);
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
