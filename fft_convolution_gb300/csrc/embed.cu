// embed.cu -- embedding of tokens and its gradient.
//
//   y_n = scale T[id_n]             (0 where id_n names no row)
//   dT[v] = scale sum of dy_n over the n with id_n = v   (+ dT[v] before)
//
// The gradient adds in one order whatever the timing: the tokens are sorted by
// row, equal rows in the order of the tokens (embed_sort_kernel), cut into
// pieces of 16 (more of many tokens) whatever the runs of equal rows are -- text
// has a few rows with a tenth of all tokens -- and summed piece by piece
// (embed_sum_kernel); runs that cross pieces leave one partial row per piece, which
// embed_join_kernel adds in the order of the pieces.
//
// Measured: 16384 tokens of 2048 bf16 columns, looked up in 20.5 us (67 MB written,
// 25 read of 6200 rows; 2 to 8 rows per thread or more blocks change nothing: it waits
// for the rows, at 27% of HBM's rate, and most of what it writes is still in the L2 when
// it ends); their gradient over 65536 rows 83 us: 268 MB of zeros with the sort beside
// them 48, which HBM bounds, the sums 22 (67 MB read and rows written), the joins 11, a
// chain of six dependent loads.
#include "cluster.cuh"
#include "seq.h"

namespace fftgb {

namespace {

// ---- lookup --------------------------------------------------------------------

__device__ __forceinline__ long long token_id(const void *ids, int id_bytes, long long n) {
  return id_bytes == 8 ? static_cast<const long long *>(ids)[n]
                       : (long long)static_cast<const int *>(ids)[n];
}

// blockDim.x threads along a row, blockDim.y rows.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) embed_kernel(const EmbedArgs a) {
  using A = typename Acc<T>::type;
  constexpr int E = VEC ? 16 / (int)sizeof(T) : 1;
  const A scale = (A)a.scale;
  const int units = a.dim / E;
  for (long long n = (long long)blockIdx.x * blockDim.y + threadIdx.y; n < a.tokens;
       n += (long long)gridDim.x * blockDim.y) {
    const long long id = token_id(a.ids, a.id_bytes, n);
    const bool there = id >= 0 && id < a.rows;
    const T *src = static_cast<const T *>(a.table) + (there ? id : 0) * a.ldt;
    T *dst = static_cast<T *>(a.y) + n * a.ldy;
#pragma unroll 4
    for (int c = threadIdx.x; c < units; c += blockDim.x) {
      if constexpr (VEC) {
        A f[E];
        uint4 w = make_uint4(0, 0, 0, 0);
        if (there) {
          unpack<T>(__ldg(reinterpret_cast<const uint4 *>(src) + c), f);
#pragma unroll
          for (int i = 0; i < E; ++i) f[i] *= scale;
          w = pack<T>(f);
        }
        reinterpret_cast<uint4 *>(dst)[c] = w;
      } else {
        dst[c] = there ? from_acc<T>(to_acc(src[c]) * scale) : from_acc<T>((A)0);
      }
    }
  }
}

// ---- tokens in the order of their rows -----------------------------------------------

constexpr int kSortMost = 16, kSortThreads = 1024, kSortBits = 9, kDigits = 1 << kSortBits;

struct SortShared {
  unsigned count[kSortThreads / 32][kDigits];  // of a tile, by warp; then where each warp's go
  unsigned base[kDigits];                      // where the next of a digit goes
  unsigned hist[kDigits];                      // of this block's tokens
  unsigned sums[kSortThreads / 32];
};

// A stable radix sort of (row, token) by one cluster of a.blocks: each block has
// its share of the tokens, digits of at most 9 bits, the arrays between the passes in
// global memory (the L2 holds them).  Tokens of no row sort behind all others.
// The clusters beside it meanwhile write zeros to the whole of a new gradient: 2
// passes over 16384 tokens hide behind 268 MB of them.
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const EmbedSortArgs a) {
  extern __shared__ __align__(16) char smem[];
  SortShared &s = *reinterpret_cast<SortShared *>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_next();
  if (blockIdx.x >= a.blocks) {
    const long long threads = (long long)(gridDim.x - a.blocks) * kSortThreads;
    const long long at = (long long)(blockIdx.x - a.blocks) * kSortThreads + tid;
    char *p = static_cast<char *>(a.fill);
    // the table's gradient starts on a boundary of its elements: 2 bytes at least
    long long head = (16 - ((uintptr_t)p & 15)) & 15;
    if (head > a.fill_bytes) head = a.fill_bytes;
    const long long words = (a.fill_bytes - head) >> 4, done = head + (words << 4);
    for (long long i = 2 * at; i < head; i += 2 * threads) *reinterpret_cast<uint16_t *>(p + i) = 0;
    for (long long i = at; i < words; i += threads)
      reinterpret_cast<uint4 *>(p + head)[i] = make_uint4(0, 0, 0, 0);
    for (long long i = done + 2 * at; i < a.fill_bytes; i += 2 * threads)
      *reinterpret_cast<uint16_t *>(p + i) = 0;
    return;
  }
  const unsigned rank = block_rank();
  if (blockIdx.x == 0 && tid == 0) *a.crossing = 0;
  const long long share = (a.tokens + a.blocks - 1) / a.blocks;
  const long long begin = min(share * rank, a.tokens), end = min(begin + share, a.tokens);
  const unsigned mask = (1u << a.bits) - 1;
  for (int d = tid; d < kDigits * (kSortThreads / 32); d += kSortThreads) (&s.count[0][0])[d] = 0;
  const int digits = 1 << a.bits;

  for (int pass = 0; pass < a.passes; ++pass) {
    const unsigned *key = a.key[pass & 1], *pos = a.pos[pass & 1];
    unsigned *key2 = a.key[(pass & 1) ^ 1], *pos2 = a.pos[(pass & 1) ^ 1];
    const int shift = pass * a.bits;
    auto key_of = [&](long long i) {
      if (pass > 0) return __ldcg(key + i);
      const long long id = token_id(a.ids, a.id_bytes, i);
      return id >= 0 && id < a.rows ? (unsigned)id : (unsigned)a.rows;
    };
    for (int d = tid; d < kDigits; d += kSortThreads) s.hist[d] = 0;
    __syncthreads();
    // whole warps: equal digits of a warp are added at once
    const unsigned first = begin + tid < end ? key_of(begin + tid) : 0;
    for (long long i0 = begin; i0 < end; i0 += kSortThreads) {
      const long long i = i0 + tid;
      const unsigned d = i < end ? ((i0 == begin ? first : key_of(i)) >> shift) & mask : ~0u;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      if (i < end && (same & ((1u << lane) - 1)) == 0) atomicAdd(&s.hist[d], (unsigned)__popc(same));
    }
    cluster_sync();
    // where this block's first token of each digit goes: behind all smaller
    // digits and the same digit of the blocks before
    unsigned total = 0, before = 0;
    if (tid < kDigits) {
      const uint32_t mine = (uint32_t)__cvta_generic_to_shared(&s.hist[tid]);
#pragma unroll
      for (unsigned r = 0; r < kSortMost; ++r)
        if (r < a.blocks) {
          const unsigned n = peer_load(peer(mine, r));
          total += n;
          if (r < rank) before += n;
        }
    }
    unsigned incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) s.sums[warp] = incl;
    __syncthreads();
    if (tid < kDigits) {
      unsigned lower = 0;
      for (int w = 0; w < warp; ++w) lower += s.sums[w];
      s.base[tid] = lower + incl - total + before;
    }
    __syncthreads();
    for (long long i0 = begin; i0 < end; i0 += kSortThreads) {
      const long long i = i0 + tid;
      const bool on = i < end;
      const unsigned k = i0 == begin ? first : on ? key_of(i) : 0;
      const unsigned p = on ? (pass > 0 ? __ldcg(pos + i) : (unsigned)i) : 0;
      const unsigned d = on ? (k >> shift) & mask : ~0u;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      const int ahead = __popc(same & ((1u << lane) - 1));
      if (on && ahead == 0) s.count[warp][d] = (unsigned)__popc(same);
      __syncthreads();
      if (tid < digits) {
        unsigned n[kSortThreads / 32], run = s.base[tid];
#pragma unroll
        for (int w = 0; w < kSortThreads / 32; ++w) n[w] = s.count[w][tid];
#pragma unroll
        for (int w = 0; w < kSortThreads / 32; ++w) {
          if (n[w] != 0) s.count[w][tid] = run;
          run += n[w];
        }
        s.base[tid] = run;
      }
      __syncthreads();
      if (on) {
        const unsigned to = s.count[warp][d] + (unsigned)ahead;
        key2[to] = k;
        pos2[to] = p;
      }
      __syncwarp();
      if (on && ahead == 0) s.count[warp][d] = 0;  // the next tile's counters, of this warp alone
    }
    __threadfence();
    cluster_sync();  // the next pass reads what every block has written; counters are free
  }
}

// ---- sums ------------------------------------------------------------------------

constexpr int kBatch = 16;  // tokens, whose rows are all loaded at once; a piece is one or more

// The columns of a warp: `E` per lane, whole 16 bytes or 32 apart.
template <typename T, bool VEC> struct Columns {
  using A = typename Acc<T>::type;
  static constexpr int E = VEC ? 16 / (int)sizeof(T) : 4;
  static constexpr int kWide = 32 * E;
  // A lane's part of a row as it lies there.
  struct alignas(VEC ? 16 : sizeof(T)) Raw {
    T v[E];
  };
  static __device__ __forceinline__ int at(int chunk, int lane, int i) {
    return chunk * kWide + (VEC ? lane * E + i : lane + 32 * i);
  }
  static __device__ __forceinline__ Raw load(const T *row, int chunk, int lane, int dim) {
    Raw r;
    if constexpr (VEC) {
      const int c = at(chunk, lane, 0);
      uint4 w = make_uint4(0, 0, 0, 0);
      if (c < dim) w = *reinterpret_cast<const uint4 *>(row + c);
      *reinterpret_cast<uint4 *>(&r) = w;
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = at(chunk, lane, i);
        r.v[i] = c < dim ? row[c] : from_acc<T>((A)0);
      }
    }
    return r;
  }
  static __device__ __forceinline__ void widen(const Raw &r, A (&f)[E]) {
    if constexpr (VEC) {
      unpack<T>(*reinterpret_cast<const uint4 *>(&r), f);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = to_acc(r.v[i]);
    }
  }
};

// A lane's part of a row of the table's gradient, of type TO (T or float):
// E columns as Columns<T, VEC> has them.
template <typename T, typename TO, bool VEC> struct Row {
  using A = typename Acc<T>::type;
  using C = Columns<T, VEC>;
  static constexpr int E = C::E;
  struct alignas(VEC ? 16 : sizeof(TO)) Raw {
    TO v[E];
  };
  static __device__ __forceinline__ TO *place(const EmbedSumArgs &a, unsigned row) {
    return static_cast<TO *>(a.dtable) + (long long)row * a.dim;
  }
  static __device__ __forceinline__ Raw load(const EmbedSumArgs &a, unsigned row, int chunk, int lane) {
    const TO *src = place(a, row);
    Raw r;
#pragma unroll
    for (int i = 0; i < E; ++i) r.v[i] = from_acc<TO>((A)0);
    if constexpr (VEC) {
      const int c = C::at(chunk, lane, 0);
      if (c < a.dim) {
#pragma unroll
        for (int j = 0; j < E * (int)sizeof(TO) / 16; ++j)
          reinterpret_cast<uint4 *>(&r)[j] = reinterpret_cast<const uint4 *>(src + c)[j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = C::at(chunk, lane, i);
        if (c < a.dim) r.v[i] = src[c];
      }
    }
    return r;
  }
  // scale f (+ old)
  static __device__ __forceinline__ void store(const EmbedSumArgs &a, unsigned row, int chunk, int lane,
                                               const A (&f)[E], const Raw *old) {
    const A scale = (A)a.scale;
    TO *dst = place(a, row);
    Raw r;
#pragma unroll
    for (int i = 0; i < E; ++i)
      r.v[i] = from_acc<TO>(old ? f[i] * scale + (A)to_acc(old->v[i]) : f[i] * scale);
    if constexpr (VEC) {
      const int c = C::at(chunk, lane, 0);
      if (c < a.dim) {
#pragma unroll
        for (int j = 0; j < E * (int)sizeof(TO) / 16; ++j)
          reinterpret_cast<uint4 *>(dst + c)[j] = reinterpret_cast<const uint4 *>(&r)[j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = C::at(chunk, lane, i);
        if (c < a.dim) dst[c] = r.v[i];
      }
    }
  }
};

// One warp per piece of the sorted tokens and chunk of columns.  ADD: rows that
// end in the piece are loaded ahead too (half a batch at a time, for the
// registers): one after the other their latency was three quarters of the time
// (5003 tokens of 1001 fp32 columns: 78 -> 9 us).
template <typename T, typename TO, bool VEC, bool ADD, bool MANY>
__global__ void __launch_bounds__(128) embed_sum_kernel(const EmbedSumArgs a) {
  using A = typename Acc<T>::type;
  using C = Columns<T, VEC>;
  using R = Row<T, TO, VEC>;
  constexpr int E = C::E, U = ADD ? kBatch / 2 : kBatch;
  let_next();
  after_previous();
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int chunks = (a.dim + C::kWide - 1) / C::kWide;
  const long long piece = item / chunks;
  const int chunk = (int)(item - piece * chunks);
  const long long first = piece * (MANY ? a.piece : kBatch);
  if (first >= a.tokens) return;
  const unsigned none = (unsigned)a.rows;
  // lanes 0 .. 15: a batch's tokens; 16: the one behind it, 17: the one before it
  auto lane_key = [&](long long at) {
    const long long where = lane < 17 ? at + lane : at - 1;
    return lane < 18 && where >= 0 && where < a.tokens ? a.key[where] : none;
  };
  auto lane_pos = [&](long long at) {
    return lane < kBatch && at + lane < a.tokens ? a.pos[at + lane] : 0u;
  };
  unsigned key = lane_key(first), pos = lane_pos(first);
  const unsigned prev = __shfl_sync(0xffffffffu, key, 17);
  const T *dy = static_cast<const T *>(a.dy);
  A *partial = static_cast<A *>(a.partial) + piece * 2 * a.ldp;
  A acc[E];
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] = 0;
  unsigned cur = __shfl_sync(0xffffffffu, key, 0);
  if (cur == none) return;  // sorted: nothing but padding from here on
  bool open = cur == prev;  // the run comes from the piece before
  // MANY: a piece of several batches (the loop and the next batch's tokens on their way
  // cost one of a single batch 2 of 22 us)
  for (int b0 = 0; b0 < (MANY ? a.piece : kBatch); b0 += kBatch) {
    const long long ahead = first + b0 + kBatch;
    const bool more = MANY && b0 + kBatch < a.piece;
    const unsigned next_key = more ? lane_key(ahead) : none, next_pos = more ? lane_pos(ahead) : 0;
#pragma unroll
    for (int j0 = 0; j0 < kBatch; j0 += U) {
      typename C::Raw f[U];
      typename R::Raw old[ADD ? U : 1];
      // the lanes hold `none` behind the last token
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const unsigned k = __shfl_sync(0xffffffffu, key, j0 + u);
        const unsigned p = __shfl_sync(0xffffffffu, pos, j0 + u);
        const bool live = k != none;
        f[u] = C::load(dy + (long long)p * a.lddy, chunk, lane, live ? a.dim : 0);
        if constexpr (ADD)
          if (live && k != __shfl_sync(0xffffffffu, key, j0 + u + 1))
            old[u] = R::load(a, k, chunk, lane);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const unsigned k = __shfl_sync(0xffffffffu, key, j0 + u);
        if (k == none) return;  // runs have been written where they end
        A v[E];
        C::widen(f[u], v);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] += v[i];
        const unsigned next = __shfl_sync(0xffffffffu, key, j0 + u + 1);
        const bool ends = next != k;
        if (!ends && (more || j0 + u + 1 < kBatch)) continue;
        // a run that begins here and goes on: one more for the joins, in any order
        if (!ends && !open && chunk == 0 && lane == 0)
          a.list[atomicAdd(a.crossing, 1u)] = (unsigned)piece;
        if (ends && !open) {
          R::store(a, k, chunk, lane, acc, ADD ? &old[ADD ? u : 0] : nullptr);
        } else {
          A *to = partial + (open ? 0 : a.ldp);
#pragma unroll
          for (int i = 0; i < E; ++i) {
            const int c = C::at(chunk, lane, i);
            if (c < a.dim) to[c] = acc[i];
          }
        }
        open = false;
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = 0;
      }
    }
    key = next_key;
    pos = next_pos;
  }
}

// The runs that go on behind the piece where they begin, from the list: its own part,
// then the heads of the pieces behind it, an equal share to each warp of the
// block (the most frequent row of a text crosses dozens; one warp for all of them, and
// blocks for every piece, took 17 us for 16384 tokens).
constexpr int kJoinWarps = 4;
template <typename T, typename TO, bool VEC>
__global__ void __launch_bounds__(32 * kJoinWarps) embed_join_kernel(const EmbedSumArgs a) {
  using A = typename Acc<T>::type;
  using C = Columns<T, VEC>;
  using R = Row<T, TO, VEC>;
  constexpr int E = C::E, U = 4;  // 8: 118 registers, 2 us more
  __shared__ A parts[kJoinWarps - 1][E][32];
  after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunks = (a.dim + C::kWide - 1) / C::kWide;
  const long long items = (long long)*a.crossing * chunks;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const long long piece = a.list[item / chunks];
    const int chunk = (int)(item % chunks);
    const unsigned row = a.key[(piece + 1) * a.piece - 1];
    long long last = piece + 1;  // the piece where the run ends: it goes on where the next begins with it
    for (;;) {
      const long long at = (last + 1 + lane) * a.piece;
      const unsigned on = __ballot_sync(0xffffffffu, at < a.tokens && a.key[at] == row);
      const int more = __ffs(~on) - 1;
      last += more < 0 ? 32 : more;
      if (more >= 0) break;
    }
    const A *partial = static_cast<const A *>(a.partial);
    A acc[E];
    typename R::Raw old;
    if (a.add && warp == 0) old = R::load(a, row, chunk, lane);
    // part 0 is the piece's own tail
    const long long count = last - piece + 1, share = (count + kJoinWarps - 1) / kJoinWarps;
    const long long from = share * warp, to = min(from + share, count);
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0;
    for (long long q = from; q < to; q += U) {
      A f[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const A *p = partial + ((piece + q + u) * 2 + (q + u == 0 ? 1 : 0)) * a.ldp;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int c = C::at(chunk, lane, i);
          f[u][i] = q + u < to && c < a.dim ? p[c] : (A)0;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] += f[u][i];
    }
    if (warp > 0) {
#pragma unroll
      for (int i = 0; i < E; ++i) parts[warp - 1][i][lane] = acc[i];
    }
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int w = 0; w < kJoinWarps - 1; ++w)
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] += parts[w][i][lane];
      R::store(a, row, chunk, lane, acc, a.add ? &old : nullptr);
    }
    __syncthreads();
  }
}

// Lets a kernel's clusters have 16 blocks, once per device and context.
cudaError_t wide_cluster_once(const void *kern, DeviceOnce &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const unsigned long long id = context_id();
  if (id != 0 && done.ctx[dev].load(std::memory_order_acquire) == id) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.ctx[dev].store(context_id(), std::memory_order_release);
  return e;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

template <typename T> cudaError_t lookup_t(const EmbedArgs &a, cudaStream_t st) {
  const bool vec = (a.dim * sizeof(T)) % 16 == 0 && (a.ldt * sizeof(T)) % 16 == 0 &&
                   (a.ldy * sizeof(T)) % 16 == 0 && aligned16(a.table) && aligned16(a.y);
  const int units = vec ? a.dim / (16 / (int)sizeof(T)) : a.dim;
  int tx = 8;  // four units of a row per thread, 8 .. 256 threads per row
  while (tx < 256 && tx * 4 < units) tx *= 2;
  const int ty = 256 / tx;
  const long long most = (long long)sm_count() * 32, need = (a.tokens + ty - 1) / ty;
  if (most <= 0) return cudaErrorInvalidDevice;
  const dim3 block(tx, ty);
  const unsigned grid = (unsigned)(need < most ? need : most);
  if (vec) embed_kernel<T, true><<<grid, block, 0, st>>>(a);
  else embed_kernel<T, false><<<grid, block, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, typename TO, bool VEC>
cudaError_t sums_t(const EmbedSumArgs &a, cudaStream_t st) {
  const long long chunks = (a.dim + Columns<T, VEC>::kWide - 1) / Columns<T, VEC>::kWide;
  const long long pieces = (a.tokens + a.piece - 1) / a.piece;
  const long long blocks = (pieces * chunks + 3) / 4;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const cudaError_t e =
      launch_kernel(true,
                    a.piece > kBatch ? (a.add ? embed_sum_kernel<T, TO, VEC, true, true>
                                              : embed_sum_kernel<T, TO, VEC, false, true>)
                                     : (a.add ? embed_sum_kernel<T, TO, VEC, true, false>
                                              : embed_sum_kernel<T, TO, VEC, false, false>),
                    (unsigned)blocks, dim3(128), 0, 1, st, a);
  if (e != cudaSuccess || pieces == 1) return e;
  const long long most = 8ll * sm_count() * 4 / kJoinWarps, items = pieces * chunks;
  return launch_kernel(true, embed_join_kernel<T, TO, VEC>, (unsigned)(items < most ? items : most),
                       dim3(32 * kJoinWarps), 0, 1, st, a);
}

template <typename T, typename TO> cudaError_t sums_to(const EmbedSumArgs &a, cudaStream_t st) {
  const bool vec = (a.dim * sizeof(T)) % 16 == 0 && (a.lddy * sizeof(T)) % 16 == 0 &&
                   (a.dim * sizeof(TO)) % 16 == 0 && aligned16(a.dy) && aligned16(a.dtable);
  return vec ? sums_t<T, TO, true>(a, st) : sums_t<T, TO, false>(a, st);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
size_t list_bytes(long long tokens) { return round256((size_t)tokens * 4); }

}  // namespace

// Tokens of a piece: many of them make long runs, whose parts one block adds (10^6
// tokens of 64 columns: 271 -> 11 us for the joins, 88 -> 104 for the sums).
int piece_tokens(long long tokens) {
  const long long batches = tokens / 32768;
  return kBatch * (int)(batches < 1 ? 1 : batches > 32 ? 32 : batches);
}

size_t embed_workspace_bytes(long long tokens, int dim, int dtype) {
  if (tokens == 0) return 0;
  const int piece = piece_tokens(tokens);
  const size_t pieces = (size_t)(tokens + piece - 1) / piece;
  return 4 * list_bytes(tokens) + 256 + list_bytes((long long)pieces) + pieces * 2 * (size_t)dim * (dtype == FFT_ELEM_F64 ? 8 : 4);
}

cudaError_t launch_embed(int dtype, const EmbedArgs &a, cudaStream_t st) {
  switch (dtype) {
    case FFT_ELEM_F32: return lookup_t<float>(a, st);
    case FFT_ELEM_F64: return lookup_t<double>(a, st);
    case FFT_ELEM_BF16: return lookup_t<__nv_bfloat16>(a, st);
    default: return lookup_t<__half>(a, st);
  }
}

cudaError_t launch_embed_grad(int dtype, int ttype, const EmbedGradArgs &g, void *workspace,
                              cudaStream_t st) {
  const size_t table_bytes = (size_t)g.rows * (size_t)g.dim * elem_bytes(ttype);
  if (g.tokens == 0)
    return g.add ? cudaSuccess : cudaMemsetAsync(g.dtable, 0, table_bytes, st);
  char *ws = static_cast<char *>(workspace);
  const size_t list = list_bytes(g.tokens);
  EmbedSortArgs s{};
  s.ids = g.ids;
  s.id_bytes = g.id_bytes;
  s.tokens = g.tokens;
  s.rows = g.rows;
  for (int i = 0; i < 2; ++i) {
    s.key[i] = reinterpret_cast<unsigned *>(ws + 2 * i * list);
    s.pos[i] = reinterpret_cast<unsigned *>(ws + (2 * i + 1) * list);
  }
  // 16 blocks from 32768 tokens on, whatever is beside the sort. Above: 65536 tokens of 1024
  // columns 130 -> 105 us (added to a table 159 -> 133), 36000 added 104 -> 91, 10^6 of 64
  // columns 955 -> 546. Below, where zeros hide the sort, they hold these back: 16384 of 2048
  // 90 -> 91, 30000 of 4096 over 65536 rows 183 -> 192. Without many zeros 8 blocks lose there
  // too: 30000 of 1024 added 77 -> 89, of 256 over 2000 rows 44 -> 52; 5003 added are even.
  s.blocks = g.tokens > 32768 ? kSortMost : 8;
  s.crossing = reinterpret_cast<unsigned *>(ws + 4 * list);
  int bits = 0;  // of the largest key, which is `rows`
  while (bits < 32 && ((unsigned long long)g.rows >> bits) != 0) ++bits;
  s.passes = (bits + kSortBits - 1) / kSortBits;
  s.bits = (bits + s.passes - 1) / s.passes;
  s.fill = g.add ? nullptr : g.dtable;
  s.fill_bytes = g.add ? 0 : (long long)table_bytes;
  // A cluster for each MB, up to four blocks per SM: 268 MB of zeros and 16384 tokens
  // take 104 us with one per SM, 88 with two, 83.5 with four, 83 with sixteen.
  long long fillers = (s.fill_bytes + (1ll << 20) - 1) >> 20;
  const long long most = 4 * (sm_count() / (int)s.blocks);
  if (fillers > most) fillers = most;
  static DeviceOnce once, wide_once;
  cudaError_t e = smem_limit_once((const void *)embed_sort_kernel, sizeof(SortShared), once);
  if (e == cudaSuccess && s.blocks > 8) e = wide_cluster_once((const void *)embed_sort_kernel, wide_once);
  if (e != cudaSuccess) return e;
  e = launch_kernel(false, embed_sort_kernel, (unsigned)(s.blocks * (1 + fillers)), dim3(kSortThreads),
                    sizeof(SortShared), s.blocks, st, s);
  if (e != cudaSuccess) return e;
  EmbedSumArgs a{};
  a.dy = g.dy;
  a.lddy = g.lddy;
  a.key = s.key[s.passes & 1];
  a.pos = s.pos[s.passes & 1];
  a.tokens = g.tokens;
  a.rows = g.rows;
  a.dim = g.dim;
  a.ldp = g.dim;
  a.piece = piece_tokens(g.tokens);
  a.crossing = s.crossing;
  a.list = reinterpret_cast<unsigned *>(ws + 4 * list + 256);
  a.partial = ws + 4 * list + 256 + list_bytes((g.tokens + a.piece - 1) / a.piece);
  a.dtable = g.dtable;
  a.scale = g.scale;
  a.add = g.add;
  switch (dtype) {
    case FFT_ELEM_F32: return sums_to<float, float>(a, st);
    case FFT_ELEM_F64: return sums_to<double, double>(a, st);
    case FFT_ELEM_BF16:
      return ttype == FFT_ELEM_F32 ? sums_to<__nv_bfloat16, float>(a, st)
                                   : sums_to<__nv_bfloat16, __nv_bfloat16>(a, st);
    default:
      return ttype == FFT_ELEM_F32 ? sums_to<__half, float>(a, st) : sums_to<__half, __half>(a, st);
  }
}

}  // namespace fftgb
