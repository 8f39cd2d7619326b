// xent.cu -- the cross entropy of a linear layer over a vocabulary, without
// its logits ever lying in memory:
//
//   l_nv = x_n . w_v,  lse_n = log sum_v e^{l_nv},  loss_n = lse_n - l_{n,t_n},
//   G_nv = c_n (e^{l_nv - lse_n} - [v = t_n]),  dx = G W,  dW = G^T x
//
// (c: the gradient of the loss; a token whose target is no word has no loss
// and no gradient).  The products are tiles of 256 tokens x 256 words on pairs of
// multiprocessors (pair_gemm.cuh).  Forward, a tile leaves each row's maximum
// and sum of exponentials, which a second kernel joins.  Backward, the logits are
// computed again from lse, piece by piece of the vocabulary: a piece's G (at
// most 256 MB, in the operands' type) is written, then both products with it run
// in one launch, dW's rows of the piece in full and dx in fp32 on top of the
// pieces before.  A product of few tiles is cut along its sum into slices, which the
// last kernel adds in order.
//
// Measured (bf16): 8192 tokens, 65536 words, 2048 wide: 1.01 ms for the sums, which is
// 2.18 PFLOP/s, 0.31 for a piece's G and 0.61 to 0.66 for its products, alone; 5.4 ms
// for the loss and its gradients (1.63 PFLOP/s of 8 N V D operations), bound by the
// power cap.  At small widths (64) the reading warps are the bound, two per scheduler:
// 44% of the issue slots, their own instructions' latencies the largest stall; the
// exponentials fill 32% of their units, the products 16% of the tensor cores.
//
// fp32 operands are laid out once per call as three bf16 parts each (24
// significand bits, any exponent), of whose nine products the six largest are
// taken: those left out are below 2^-24 of the factors' sizes.
#include <math.h>

#include "pair_gemm.cuh"
#include "tensor_map.h"

namespace fftgb {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr size_t kPieceBytes = (size_t)256 << 20;  // of G

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ long long target_of(const void *t, int bytes, long long n) {
  return bytes == 8 ? static_cast<const long long *>(t)[n]
                    : (long long)static_cast<const int *>(t)[n];
}

// ---- operands ---------------------------------------------------------------------

// Which rows count: those of tokens with a target and a weight (null: all).
struct LiveRows {
  const void *targets;
  int target_bytes;
  long long vocabulary;
  const float *dloss;
};
// One operand: rows of ld elements, `vec`: on boundaries of 16 bytes.
template <typename T, typename O> struct LayRows {
  const T *in;
  long long ld, rows;
  O *out;
  int ldo;
  bool vec;
};
// Rows as `PARTS` arrays of rows of ldo elements, whole 16 bytes; those of x that do not
// count are 0.  x and W in one launch (either may have no rows); a thread makes
// eight elements at a time.
template <typename T, typename O, int PARTS>
__global__ void __launch_bounds__(256) xent_lay_kernel(const LayRows<T, O> x, const LayRows<T, O> w,
                                                       int dim, LiveRows live) {
  let_next();
  for (long long at = (long long)blockIdx.x * blockDim.y + threadIdx.y; at < x.rows + w.rows;
       at += (long long)gridDim.x * blockDim.y) {
    const bool mine = at < x.rows;
    const LayRows<T, O> &o = mine ? x : w;
    const long long r = mine ? at : at - x.rows;
    int wide = dim;
    if (mine && live.targets) {
      const long long t = target_of(live.targets, live.target_bytes, r);
      if (t < 0 || t >= live.vocabulary || live.dloss[r] == 0.0f) wide = 0;
    }
#pragma unroll 4
    for (int c = 8 * threadIdx.x; c < o.ldo; c += 8 * blockDim.x) {
      const T *src = o.in + r * o.ld + c;
      O *dst = o.out + r * o.ldo + c;
      if constexpr (PARTS == 1) {
        alignas(16) T v[8];
        if (o.vec && c + 8 <= wide) {
          *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(src);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = c + i < wide ? src[i] : from_acc<T>(0.0f);
        }
        *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(v);
      } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < wide ? src[i] : 0.0f;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
          float h[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            h[i] = to_acc(from_acc<O>(v[i]));
            // float's largest values round to infinity: cut off instead
            if (isinf(h[i]) && isfinite(v[i])) h[i] = __uint_as_float(__float_as_uint(v[i]) & 0xffff0000u);
            v[i] = isfinite(h[i]) ? v[i] - h[i] : 0.0f;
          }
          *reinterpret_cast<uint4 *>(dst + (long long)p * o.rows * o.ldo) = pack<O>(h);
        }
      }
    }
  }
}

// ---- forward ----------------------------------------------------------------------

struct XentTiles {
  long long tokens, vocabulary;
  int m, n;  // tiles of tokens and of words
  const void *targets;
  int target_bytes;
  int width;  // words of a tile (few tokens: tokens)
  int part;   // words of a part
  // forward: per half a tile's words and token, largest logit and sum (both in powers of 2)
  float2 *partial;
  float *at_target;
  // gradient: a piece of the words from v0 on
  long long v0;
  const float *lse, *dloss;
  const float *unit;  // what G is scaled by (null: 1)
  void *g;            // [parts][tokens][ldg]
  long long ldg;
};

constexpr int kHalf = kPairTile / 2;  // columns of a lane, at most

constexpr int kFewTokens = 128;  // up to here words are the rows of a tile

// Tiles of all token blocks before the next words: x stays in the L2, W is read once.
__device__ __forceinline__ PairTile word_tile(const XentTiles &p, int t, long long v0, int k) {
  PairTile w{};
  w.a_row = (t % p.m) * kPairTile;
  w.b_row = (int)v0 + (t / p.m) * p.width;
  w.k0 = 0;
  w.k1 = k;
  return w;
}

__global__ void __launch_bounds__(kPairThreads, 1)
xent_sums_kernel(const __grid_constant__ PairOperands ops, const XentTiles p, int kblocks,
                 int *status) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)block_rank(), half = (warp - 4) >> 2;
  auto of = [&](int t, int &) { return word_tile(p, t, 0, kblocks); };
  auto out = [&](int t, float (&f)[kHalf]) {
    const PairTile w = word_tile(p, t, 0, kblocks);
    const long long n = w.a_row + rank * 128 + (warp & 3) * 32 + lane;
    const int wide = p.width / 2;
    const long long v0 = w.b_row + half * wide;
    if (v0 >= p.vocabulary || n >= p.tokens) return;
    const int count = (int)min((long long)wide, p.vocabulary - v0);
    const long long target = target_of(p.targets, p.target_bytes, n) - v0;
    const bool mine = target >= 0 && target < count;
    if (mine) {
      float at = 0.0f;
#pragma unroll
      for (int i = 0; i < kHalf; ++i)
        if (target == i) at = f[i];
      p.at_target[n] = at;
    }
    if (count < wide) {  // the last words: what is behind them does not count
#pragma unroll
      for (int i = 0; i < kHalf; ++i)
        if (i >= count) f[i] = -INFINITY;
    }
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kHalf; j += 32)
      if (j < wide) {
#pragma unroll
        for (int i = 0; i < 32; ++i) top = fmaxf(top, f[j + i]);
      }
    // all of them -infinity (or NaN): in units of 1
    top = top == -INFINITY ? top : top * kLog2e;
    const float unit = top == -INFINITY ? 0.0f : top;
    float2 sums = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < kHalf; j += 32)
      if (j < wide) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 e = fma2(make_float2(f[j + i], f[j + i + 1]), both(kLog2e), both(-unit));
          sums = add2(sums, make_float2(exp2_approx(e.x), exp2_approx(e.y)));
        }
      }
    const float sum = sums.x + sums.y;
    p.partial[(2ll * (t / p.m) + half) * p.tokens + n] = make_float2(sum == 0.0f ? top : unit, sum);
  };
  pair_run(&ops, p.m * p.n, status, of, out);
}

// The same for few tokens: tiles of 256 words x up to 128 tokens, so that a stage holds
// little but words (W is all there is to read: 48 tokens, 65536 words, 4096 wide 105
// -> 98 us).  A lane's row is a word: 32 x 32 logits at a time turn in shared memory, after
// which a lane has one token's.  Parts are of 32 words.
__global__ void __launch_bounds__(kPairThreads, 1)
xent_few_kernel(const __grid_constant__ PairOperands ops, const XentTiles p, int kblocks, int *status) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)block_rank(), half = (warp - 4) >> 2;
  auto of = [&](int t, int &) {
    PairTile w{};
    w.a_row = t * kPairTile;
    w.k1 = kblocks;
    return w;
  };
  auto out = [&](int t, float (&f)[kHalf]) {
    const long long v0 = (long long)t * kPairTile + rank * 128 + (warp & 3) * 32;
    if (v0 >= p.vocabulary) return;
    const int count = (int)min(32ll, p.vocabulary - v0);
    float *turn = pair_spare() + (warp - 4) * (32 * 33);
    const int wide = p.width / 2;
#pragma unroll
    for (int j = 0; j < kHalf; j += 32)
      if (j < wide && half * wide + j < p.tokens) {
#pragma unroll
        for (int i = 0; i < 32; ++i) turn[i * 33 + lane] = f[j + i];
        __syncwarp();
        const long long n = half * wide + j + lane;
        if (n < p.tokens) {
          const float *l = turn + lane * 33;
          const long long target = target_of(p.targets, p.target_bytes, n) - v0;
          if (target >= 0 && target < count) p.at_target[n] = l[target];
          float top = -INFINITY, sum = 0.0f;
          for (int i = 0; i < count; ++i) top = fmaxf(top, l[i]);
          // all of them -infinity (or NaN): in units of 1
          top = top == -INFINITY ? top : top * kLog2e;
          const float unit = top == -INFINITY ? 0.0f : top;
          for (int i = 0; i < count; ++i) sum += exp2_approx(fmaf(l[i], kLog2e, -unit));
          p.partial[(v0 >> 5) * p.tokens + n] = make_float2(sum == 0.0f ? top : unit, sum);
        }
        __syncwarp();
      }
  };
  pair_run(&ops, p.n, status, of, out);
}

// (m, s) + (m', s'): the sums in units of the larger power of two.
__device__ __forceinline__ float2 join_sums(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  const float sa = a.x == m ? a.y : a.y * exp2f(a.x - m), sb = b.x == m ? b.y : b.y * exp2f(b.x - m);
  return make_float2(m, sa + sb);
}
// lse and loss from the parts of a token: blocks of T tokens, the parts of each taken
// by blockDim.x / T threads (with 32 tokens and every eighth part, 48 tokens of 512 parts
// took 16 us; with 8 tokens and every 128th, 65536 tokens of 8 parts 100).
template <int T>
__global__ void __launch_bounds__(1024) xent_join_kernel(const XentTiles p, float *loss, float *lse) {
  __shared__ float2 parts[1024];
  after_previous();
  const int at = threadIdx.x % T, slice = threadIdx.x / T, slices = blockDim.x / T;
  const long long n = (long long)blockIdx.x * T + at;
  const int count = (int)((p.vocabulary + p.part - 1) / p.part);
  float2 s = make_float2(-INFINITY, 0.0f);
  if (n < p.tokens) {
#pragma unroll 4
    for (int i = slice; i < count; i += slices)
      s = join_sums(s, p.partial[(long long)i * p.tokens + n]);
  }
  parts[threadIdx.x] = s;
  for (int half = slices / 2; half > 0; half /= 2) {
    __syncthreads();
    if (slice < half) {
      s = join_sums(s, parts[threadIdx.x + half * T]);
      parts[threadIdx.x] = s;
    }
  }
  if (slice > 0 || n >= p.tokens) return;
  const float total = (s.x + log2f(s.y)) * kLn2;
  const long long target = target_of(p.targets, p.target_bytes, n);
  lse[n] = total;
  loss[n] = target >= 0 && target < p.vocabulary ? total - p.at_target[n] : 0.0f;
}

// ---- gradients ----------------------------------------------------------------------

// For half operands: the power of two that brings the largest |c_n| to 2^14 ..
// 2^15, so that G = c (p - 1) uses the type's range, and its inverse.
__global__ void __launch_bounds__(1024) xent_unit_kernel(const XentTiles p, float *unit) {
  __shared__ float most[32];
  let_next();
  after_previous();
  float m = 0.0f;
  for (long long n = threadIdx.x; n < p.tokens; n += 1024) {
    const long long t = target_of(p.targets, p.target_bytes, n);
    if (t >= 0 && t < p.vocabulary) m = fmaxf(m, fabsf(p.dloss[n]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < 32; ++w) m = fmaxf(m, most[w]);
  int e = 0;
  float u = 1.0f;
  if (m > 0.0f && isfinite(m)) {
    frexpf(m, &e);  // m < 2^e
    u = ldexpf(1.0f, min(max(15 - e, -100), 100));
  }
  unit[0] = u;
  unit[1] = 1.0f / u;
}

__device__ __forceinline__ void store32(void *p, uint4 a, uint4 b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y),
               "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}
// 32 values as PARTS arrays, in stores of 32 bytes, a whole sector of a row each.
template <typename O, int PARTS>
__device__ __forceinline__ void put32(O *row, long long part, float (&f)[32]) {
#pragma unroll
  for (int q = 0; q < PARTS; ++q) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint4 w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[16 * j + 8 * h + i];
        w[h] = pack<O>(v);
        if constexpr (PARTS > 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[16 * j + 8 * h + i] -= to_acc(from_acc<O>(v[i]));
        }
      }
      store32(row + q * part + 16 * j, w[0], w[1]);
    }
  }
}

// G of a piece of the vocabulary; columns behind the last word are 0.  Rounded to 16
// bits for the products it takes part in (dx and dw of 16-bit operands come out
// 2.4e-3 off in the mean where one rounding at the end gives 1.7e-3); float
// operands get all of it.
template <typename O, int PARTS>
__global__ void __launch_bounds__(kPairThreads, 1)
xent_grad_kernel(const __grid_constant__ PairOperands ops, const XentTiles p, int kblocks,
                 int *status) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)block_rank(), half = (warp - 4) >> 2;
  auto of = [&](int t, int &) { return word_tile(p, t, p.v0, kblocks); };
  auto out = [&](int t, float (&f)[kHalf]) {
    const PairTile w = word_tile(p, t, p.v0, kblocks);
    const long long n = w.a_row + rank * 128 + (warp & 3) * 32 + lane;
    const int wide = p.width / 2;
    const long long v = w.b_row + half * wide;
    // a token that takes no part: e^{0 - infinity} * 0 (its x has been laid out as 0)
    float c = 0.0f, lse = INFINITY;
    int at = -1;
    if (n < p.tokens) {
      const long long target = target_of(p.targets, p.target_bytes, n);
      if (target >= 0 && target < p.vocabulary && p.dloss[n] != 0.0f) {
        c = p.dloss[n] * (p.unit ? p.unit[0] : 1.0f);
        lse = p.lse[n];
        if (target >= v && target < v + wide) at = (int)(target - v);
      }
    }
    O *row = static_cast<O *>(p.g) + n * p.ldg + (v - p.v0);
    const int count = (int)max(0ll, min((long long)wide, p.vocabulary - v));
#pragma unroll
    for (int j = 0; j < kHalf; j += 32)
      if (j < wide) {
        float q[32];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          // l - lse is exact where it counts, near 0: a product with log2 e before it would round lse
          const float2 l = add2(make_float2(f[j + i], f[j + i + 1]), both(-lse));
          const float2 e = mul2(l, both(kLog2e));
          q[i] = exp2_approx(e.x);
          q[i + 1] = exp2_approx(e.y);
        }
        if (__any_sync(0xffffffffu, at >= j && at < j + 32)) {
#pragma unroll
          for (int i = 0; i < 32; ++i) q[i] -= at == j + i ? 1.0f : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 g = mul2(make_float2(q[i], q[i + 1]), both(c));
          q[i] = g.x;
          q[i + 1] = g.y;
        }
        if (count < wide) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (j + i >= count) q[i] = 0.0f;
        }
        if (n < p.tokens) put32<O, PARTS>(row + j, p.tokens * p.ldg, q);
      }
  };
  pair_run(&ops, p.m * p.n, status, of, out);
}

// dx += G W over a piece and dW = G^T x of its rows, in one launch: the
// longer sums first, so that the short ones fill the ends.
struct XentProducts {
  PairOperands ops[2];
  long long tokens, v0;
  long long words;       // of the piece
  int dim;
  int width;             // columns of a tile
  int m, n, slices, k;   // dx: tiles of tokens and of columns, cuts of the sum, its blocks
  int wm, wk, wslices;   // dW: tiles of words, blocks of tokens, cuts of their sum
  int words_first;       // dW's tiles before dx's
  float *wsums;          // [wslices][words][dim]; one cut: not used
  float *sums;           // [slices][tokens][dim]
  int first;             // the piece: nothing to add to
  void *dw;
  void *dx;              // one piece and one cut: the result; else null
  const float *unit;
};

// Adds to four floats where they lie: a reduction in the L2, once per element and launch,
// that nobody waits for (to load, add and store them held the products back).
__device__ __forceinline__ void add16(float *p, const float (&v)[4]) {
  asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3])
               : "memory");
}
// 32 columns from c on of a warp's 32 rows (a lane has one) into an array of rows of
// dim elements, + what is there (floats only).  Rows on 32-byte boundaries: each lane its own;
// others: a row at a time, through shared memory (each lane writing its row by
// elements took half the time of 777 tokens, 333 wide).
template <typename T>
__device__ __forceinline__ void put_rows(T *out, long long row0, long long rows, int c, int dim, bool vec,
                                         bool add, float (&f)[32], float *turn) {
  constexpr int P = 16 / (int)sizeof(T);
  const int lane = threadIdx.x & 31;
  if (vec) {
    if (row0 + lane >= rows) return;
    T *row = out + (row0 + lane) * dim + c;
#pragma unroll
    for (int j = 0; j < 32; j += 2 * P) {
      if (c + j < dim) {
        uint4 w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[P];
#pragma unroll
          for (int i = 0; i < P; ++i) v[i] = f[j + h * P + i];
          if constexpr (sizeof(T) == 4)
            if (add) {
              add16(row + j + h * P, v);
              continue;
            }
          w[h] = pack<T>(v);
        }
        if (!add) store32(row + j, w[0], w[1]);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) turn[lane * 33 + i] = f[i];
  __syncwarp();
  const int count = (int)max(0ll, min(32ll, rows - row0));
  if (c + lane < dim) {
    T *col = out + row0 * dim + c + lane;
#pragma unroll 8
    for (int r = 0; r < count; ++r) {
      const float v = turn[r * 33 + lane];
      if constexpr (sizeof(T) == 4)
        if (add) {
          atomicAdd(col + (long long)r * dim, v);
          continue;
        }
      col[(long long)r * dim] = from_acc<T>(v);
    }
  }
  __syncwarp();
}

template <typename T>
__global__ void __launch_bounds__(kPairThreads, 1)
xent_products_kernel(const __grid_constant__ XentProducts p, int *status) {
  const int warp = threadIdx.x >> 5;
  const int rank = (int)block_rank(), half = (warp - 4) >> 2;
  const int mn = p.m * p.n, dx_tiles = mn * p.slices;
  const int wmn = p.wm * p.n, dw_tiles = wmn * p.wslices;
  // which of the products (0: dx), which cut, and the tile there
  auto place = [&](int t, int &which, int &slice) {
    int u = p.words_first ? (t < dw_tiles ? t + dx_tiles : t - dw_tiles) : t;
    which = u < dx_tiles ? 0 : 1;
    if (which) u -= dx_tiles;
    slice = u / (which ? wmn : mn);
    return u - slice * (which ? wmn : mn);
  };
  auto of = [&](int t, int &which) {
    PairTile w{};
    int slice;
    const int u = place(t, which, slice);
    const long long k = which ? p.wk : p.k;
    const int slices = which ? p.wslices : p.slices;
    w.a_row = u / p.n * kPairTile;
    w.b_row = u % p.n * p.width;
    w.b_base = which ? 0 : (int)p.v0;
    w.k0 = (int)(k * slice / slices);
    w.k1 = (int)(k * (slice + 1) / slices);
    return w;
  };
  auto out = [&](int t, float (&f)[kHalf]) {
    int which, slice;
    place(t, which, slice);
    const PairTile w = of(t, which);
    const long long r0 = w.a_row + rank * 128 + (warp & 3) * 32;  // the warp's first row
    const int wide = p.width / 2, c0 = w.b_row + half * wide;
    const bool last = which ? p.wslices == 1 : p.dx != nullptr;  // the result, not a part of it
    const float back = last && p.unit ? p.unit[1] : 1.0f;
    float *turn = pair_spare() + (warp - 4) * (32 * 33);
#pragma unroll
    for (int j = 0; j < kHalf; j += 32)
      if (j < wide && c0 + j < p.dim) {
        float q[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) q[i] = f[j + i] * back;
        const int c = c0 + j;
        if (!last) {
          const long long rows = which ? p.words : p.tokens;
          put_rows<float>((which ? p.wsums : p.sums) + slice * rows * p.dim, r0, rows, c, p.dim,
                          p.dim % 8 == 0, which == 0 && !p.first, q, turn);
        } else {
          T *out = which ? static_cast<T *>(p.dw) + p.v0 * p.dim : static_cast<T *>(p.dx);
          const bool vec = p.dim * (int)sizeof(T) % 32 == 0 && ((uintptr_t)out & 31) == 0;
          put_rows<T>(out, r0, which ? p.words : p.tokens, c, p.dim, vec, false, q, turn);
        }
      }
  };
  pair_run(p.ops, dx_tiles + dw_tiles, status, of, out);
}

// dx (dW of few words): the slices added and rounded once.
template <typename T>
__global__ void __launch_bounds__(256) xent_slices_kernel(const float *sums, long long count, int slices,
                                                      const float *unit, T *dx, bool vec) {
  after_previous();
  const float back = unit ? unit[1] : 1.0f;
  const long long step = (long long)gridDim.x * 256, first = (long long)blockIdx.x * 256 + threadIdx.x;
  if (vec) {
    for (long long i = first; i < count / 4; i += step) {
      float4 s = reinterpret_cast<const float4 *>(sums)[i];
      for (int k = 1; k < slices; ++k) {
        const float4 o = *reinterpret_cast<const float4 *>(sums + k * count + 4 * i);
        s.x += o.x;
        s.y += o.y;
        s.z += o.z;
        s.w += o.w;
      }
      T *d = dx + 4 * i;
      if constexpr (sizeof(T) == 2) {
        const T v[4] = {from_acc<T>(s.x * back), from_acc<T>(s.y * back), from_acc<T>(s.z * back),
                        from_acc<T>(s.w * back)};
        uint2 u;
        memcpy(&u, v, 8);
        *reinterpret_cast<uint2 *>(d) = u;
      } else {
        *reinterpret_cast<float4 *>(d) = make_float4(s.x * back, s.y * back, s.z * back, s.w * back);
      }
    }
    return;
  }
  for (long long i = first; i < count; i += step) {
    float s = sums[i];
    for (int k = 1; k < slices; ++k) s += sums[k * count + i];
    dx[i] = from_acc<T>(s * back);
  }
}

// ---- host -----------------------------------------------------------------------------

// [parts][rows][cols] at a row stride of ld elements, boxes of 64 columns and
// `box` rows; what lies outside reads as 0.
bool make_map(CUtensorMap *map, bool half, const void *p, long long rows, long long cols,
              long long ld, int parts, int box) {
  const TensorMapEncodeFn fn = tensor_map_encode();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)parts};
  // one part has no stride between parts, whatever its size
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * (cuuint64_t)(parts > 1 ? rows : 1)};
  const cuuint32_t shape[3] = {64, (cuuint32_t)box, 1}, ones[3] = {1, 1, 1};
  return fn(map, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<void *>(p), dims, strides, shape, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint32_t idesc_of(bool half, int width, bool a_mn, bool b_mn) {
  return mma_desc(kPairTile, width, a_mn, b_mn) | (half ? 0u : (1u << 7) | (1u << 10));
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
long long up(long long n, long long d) { return (n + d - 1) / d; }
char *first_boundary(void *workspace) {
  return reinterpret_cast<char *>(((uintptr_t)workspace + 255) & ~(uintptr_t)255);
}

// An operand as the loads can take it: the caller's array, or laid out in the workspace.
struct Operand {
  bool own;
  long long ld;
  size_t bytes;  // in the workspace
};
Operand operand(int dtype, const void *p, long long ld, long long rows, int dim, bool copy) {
  Operand o{};
  const int parts = dtype == FFT_ELEM_F32 ? 3 : 1;
  o.own = copy || parts > 1 || ((uintptr_t)p & 15) != 0 || (ld * 2) % 16 != 0;
  o.ld = o.own ? up(dim, 8) * 8 : ld;
  o.bytes = o.own ? round256((size_t)parts * rows * o.ld * 2) : 0;
  return o;
}

// Words per tile: the width that takes the pairs the least time, in rounds of all of
// them, where a tile costs as much as 32 columns beside its own (its first loads; at
// many rounds that leaves 256).  777 tokens of 10007 words: 63 -> 52 us for G in fp32.
int tile_width(long long words, long long m) {
  const long long pairs = sm_count() > 1 ? sm_count() / 2 : 1;
  long long best = 0, least = 0;
  for (int width = kPairTile; width >= 64; width -= 64) {
    const long long cost = up(m * up(words, width), pairs) * (width + 32);
    if (best == 0 || cost < least) {
      best = width;
      least = cost;
    }
  }
  return (int)best;
}

// Where everything lies, from the workspace's first 256-byte boundary on: G and the float
// sums are stored 32 bytes at a time, and a caller's workspace is on 16.
struct Layout {
  Operand x, w;
  int parts;
  size_t partial, at_target;         // forward
  bool few;
  int part;                          // words of a part of lse
  int width, wide;                   // words and columns of dx and dw per tile
  long long piece;                   // words
  int pieces, slices;
  int wslices;
  size_t unit, g, sums, wsums;       // backward
  size_t bytes;
  Layout(int dtype, const XentArgs &a, bool grad) {
    parts = dtype == FFT_ELEM_F32 ? 3 : 1;
    // gradients: x without the rows that do not count, whatever they hold (66 MB
    // moved before 4 * 10^12 operations of the largest case)
    x = operand(dtype, a.x, a.ldx, a.tokens, a.dim, grad);
    w = operand(dtype, a.w, a.ldw, a.vocabulary, a.dim, false);
    bytes = x.bytes + w.bytes;
    few = !grad && a.tokens <= kFewTokens;
    width = few ? (int)up(a.tokens, 64) * 64 : tile_width(a.vocabulary, up(a.tokens, kPairTile));
    part = few ? 32 : width / 2;
    // columns: as few tiles as there are of 256, of even size
    wide = (int)up(up(a.dim, up(a.dim, kPairTile)), 64) * 64;
    partial = at_target = unit = g = sums = wsums = 0;
    piece = 0;
    pieces = slices = wslices = 0;
    auto take = [&](size_t n) {
      const size_t at = bytes;
      bytes += round256(n);
      return at;
    };
    if (!grad) {
      partial = take((size_t)up(a.vocabulary, part) * a.tokens * 8);
      at_target = take((size_t)a.tokens * 4);
      return;
    }
    const long long words = up(a.vocabulary, width);
    long long fit = (long long)(kPieceBytes / ((size_t)a.tokens * 2 * parts * width));
    // 1024 words at least: dx is read and written once per piece
    if (fit * width < 1024) fit = up(1024, width);
    pieces = (int)up(words, fit);
    piece = up(words, pieces) * width;
    // dx's sums are cut so that its tiles fill the pairs, into cuts of 16 blocks at least
    const long long tiles = up(a.tokens, kPairTile) * up(a.dim, wide);
    const long long pairs = sm_count() > 1 ? sm_count() / 2 : 1;
    slices = 1;
    while (slices < 32 && tiles * slices * 2 <= pairs && piece / kPairK / (slices * 2) >= 16)
      slices *= 2;
    // and so are dW's, of few words and many tokens
    const long long wtiles = up(piece, kPairTile) * up(a.dim, wide);
    wslices = 1;
    while (wslices < 32 && wtiles * wslices * 2 <= pairs && up(a.tokens, kPairK) / (wslices * 2) >= 16)
      wslices *= 2;
    unit = take(8);
    g = take((size_t)parts * a.tokens * piece * 2);
    if (pieces > 1 || slices > 1) sums = take((size_t)slices * a.tokens * a.dim * 4);
    if (wslices > 1) wsums = take((size_t)wslices * piece * a.dim * 4);
  }
};

template <auto Kern, typename... Args>
cudaError_t pair_launch(bool chained, long long tiles, cudaStream_t st, const Args &...args) {
  static DeviceOnce once;
  cudaError_t e = smem_limit_once((const void *)Kern, kPairSmem, once);
  if (e != cudaSuccess) return e;
  // the split of registers counts on what a block is launched with
  static std::atomic<int> regs;
  if (regs.load(std::memory_order_acquire) == 0) {
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, (const void *)Kern);
    if (e != cudaSuccess) return e;
    regs.store(at.numRegs, std::memory_order_release);
  }
  if (regs.load(std::memory_order_acquire) < kPairRegs) return cudaErrorLaunchOutOfResources;
  const long long pairs = sm_count() / 2;
  return launch_kernel(chained, Kern, (unsigned)(2 * (tiles < pairs ? tiles : pairs)),
                       dim3(kPairThreads), kPairSmem, 2, st, args...);
}

// The type of the products' operands.
template <typename T> struct Part { using type = T; };
template <> struct Part<float> { using type = __nv_bfloat16; };

// Lays out what has to be; xp, wp: the operands.
template <typename T>
cudaError_t lay_both(const XentArgs &a, const Layout &l, char *ws, bool grad, const void *&xp,
                     const void *&wp, cudaStream_t st) {
  using O = typename Part<T>::type;
  xp = l.x.own ? ws : a.x;
  wp = l.w.own ? ws + l.x.bytes : a.w;
  if (!l.x.own && !l.w.own) return cudaSuccess;
  const LiveRows all{}, live{a.targets, a.target_bytes, a.vocabulary, a.dloss};
  auto rows = [](const void *in, long long ld, long long n, const Operand &o, char *out) {
    return LayRows<T, O>{static_cast<const T *>(in), ld, o.own ? n : 0, reinterpret_cast<O *>(out),
                         (int)o.ld, ((uintptr_t)in & 15) == 0 && ld % 8 == 0};
  };
  const LayRows<T, O> x = rows(a.x, a.ldx, a.tokens, l.x, ws);
  const LayRows<T, O> w = rows(a.w, a.ldw, a.vocabulary, l.w, ws + l.x.bytes);
  const int tx = a.dim >= 512 ? 64 : 16;
  const long long need = up(x.rows + w.rows, 256 / tx), most = (long long)sm_count() * 16;
  return launch_kernel(false, xent_lay_kernel<T, O, sizeof(T) == 4 ? 3 : 1>,
                       (unsigned)(need < most ? need : most), dim3(tx, 256 / tx), 0, 1, st, x, w, a.dim,
                       grad ? live : all);
}

template <typename T>
cudaError_t add_slices(const float *sums, long long count, int slices, const float *unit, T *out,
                       cudaStream_t st) {
  const bool vec = count % 4 == 0 && ((uintptr_t)out & (4 * sizeof(T) - 1)) == 0;
  const long long need = up(vec ? count / 4 : count, 256), most = (long long)sm_count() * 16;
  return launch_kernel(true, xent_slices_kernel<T>, (unsigned)(need < most ? need : most), dim3(256), 0,
                       1, st, sums, count, slices, unit, out, vec);
}

XentTiles tiles_of(const XentArgs &a) {
  XentTiles t{};
  t.tokens = a.tokens;
  t.vocabulary = a.vocabulary;
  t.m = (int)up(a.tokens, kPairTile);
  t.targets = a.targets;
  t.target_bytes = a.target_bytes;
  t.lse = a.lse;
  t.dloss = a.dloss;
  return t;
}

template <typename T>
cudaError_t xent_t(int dtype, const XentArgs &a, char *ws, cudaStream_t st) {
  constexpr bool half = std::is_same<T, __half>::value;
  int *status = device_status_word();
  if (!status) return cudaErrorInvalidDevice;
  const Layout l(dtype, a, false);
  const void *xp, *wp;
  cudaError_t e = lay_both<T>(a, l, ws, false, xp, wp, st);
  if (e != cudaSuccess) return e;
  PairOperands ops{};
  if (!make_map(l.few ? &ops.b : &ops.a, half, xp, a.tokens, a.dim, l.x.ld, l.parts,
                l.few ? l.width / 2 : 128) ||
      !make_map(l.few ? &ops.a : &ops.b, half, wp, a.vocabulary, a.dim, l.w.ld, l.parts,
                l.few ? 128 : l.width / 2))
    return cudaErrorInvalidValue;
  ops.width = l.width;
  ops.b_bytes = (uint32_t)l.width / 2 * 128;
  ops.idesc = idesc_of(half, l.width, false, false);
  ops.parts = l.parts;
  ops.waits = waits_now();
  XentTiles t = tiles_of(a);
  t.width = l.width;
  t.part = l.part;
  t.n = (int)up(a.vocabulary, l.few ? kPairTile : l.width);
  t.partial = reinterpret_cast<float2 *>(ws + l.partial);
  t.at_target = reinterpret_cast<float *>(ws + l.at_target);
  const int kblocks = (int)up(a.dim, kPairK);
  const bool laid = l.x.own || l.w.own;
  e = l.few ? pair_launch<xent_few_kernel>(laid, t.n, st, ops, t, kblocks, status)
            : pair_launch<xent_sums_kernel>(laid, (long long)t.m * t.n, st, ops, t, kblocks, status);
  if (e != cudaSuccess) return e;
  const long long parts = up(a.vocabulary, l.part);
  if (a.tokens <= 8ll * sm_count() && parts > 32)
    return launch_kernel(true, xent_join_kernel<8>, (unsigned)up(a.tokens, 8), dim3(1024), 0, 1, st, t,
                         a.loss, a.lse);
  int threads = 32;  // 4 parts a thread, 1 to 32 threads a token
  while (threads < 1024 && threads / 32 * 4 < parts) threads *= 2;
  return launch_kernel(true, xent_join_kernel<32>, (unsigned)up(a.tokens, 32), dim3(threads), 0, 1, st,
                       t, a.loss, a.lse);
}

template <typename T>
cudaError_t xent_grad_t(int dtype, const XentArgs &a, char *ws, cudaStream_t st) {
  using O = typename Part<T>::type;
  constexpr bool half = std::is_same<T, __half>::value;
  constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
  int *status = device_status_word();
  if (!status) return cudaErrorInvalidDevice;
  const Layout l(dtype, a, true);
  const void *xp, *wp;
  cudaError_t e = lay_both<T>(a, l, ws, true, xp, wp, st);
  if (e != cudaSuccess) return e;
  XentTiles t = tiles_of(a);
  t.width = l.width;
  float *unit = nullptr;
  if (half) {
    unit = reinterpret_cast<float *>(ws + l.unit);
    e = launch_kernel(true, xent_unit_kernel, 1, dim3(1024), 0, 1, st, t, unit);
    if (e != cudaSuccess) return e;
  }
  t.unit = unit;
  t.g = ws + l.g;
  t.ldg = l.piece;
  PairOperands ops{};
  XentProducts p{};
  if (!make_map(&ops.a, half, xp, a.tokens, a.dim, l.x.ld, l.parts, 128) ||
      !make_map(&ops.b, half, wp, a.vocabulary, a.dim, l.w.ld, l.parts, l.width / 2) ||
      !make_map(&p.ops[0].a, half, t.g, a.tokens, l.piece, l.piece, l.parts, 128) ||
      !make_map(&p.ops[0].b, half, wp, a.vocabulary, a.dim, l.w.ld, l.parts, 64) ||
      !make_map(&p.ops[1].a, half, t.g, a.tokens, l.piece, l.piece, l.parts, 64) ||
      !make_map(&p.ops[1].b, half, xp, a.tokens, a.dim, l.x.ld, l.parts, 64))
    return cudaErrorInvalidValue;
  ops.width = l.width;
  ops.b_bytes = (uint32_t)l.width / 2 * 128;
  p.width = p.ops[0].width = p.ops[1].width = l.wide;
  p.ops[0].b_bytes = p.ops[1].b_bytes = (uint32_t)up(l.wide / 2, 64) * 64 * 128;
  ops.idesc = idesc_of(half, l.width, false, false);
  p.ops[0].b_mn = p.ops[1].a_mn = p.ops[1].b_mn = 1;
  p.ops[0].idesc = idesc_of(half, l.wide, false, true);
  p.ops[1].idesc = idesc_of(half, l.wide, true, true);
  ops.parts = p.ops[0].parts = p.ops[1].parts = l.parts;
  ops.waits = p.ops[0].waits = waits_now();
  p.tokens = a.tokens;
  p.dim = a.dim;
  p.m = t.m;
  p.n = (int)up(a.dim, l.wide);
  p.slices = a.dx ? l.slices : 0;
  p.wk = (int)up(a.tokens, kPairK);
  p.wslices = l.wslices;
  p.sums = reinterpret_cast<float *>(ws + l.sums);
  p.wsums = reinterpret_cast<float *>(ws + l.wsums);
  p.dw = a.dw;
  p.dx = l.pieces == 1 && l.slices == 1 ? a.dx : nullptr;
  p.unit = unit;
  const int kblocks = (int)up(a.dim, kPairK);
  for (int i = 0; i < l.pieces; ++i) {
    t.v0 = p.v0 = i * l.piece;
    if (t.v0 >= a.vocabulary) break;
    const long long words = a.vocabulary - t.v0 < l.piece ? a.vocabulary - t.v0 : l.piece;
    t.n = (int)up(words, l.width);
    e = pair_launch<xent_grad_kernel<O, kParts>>(true, (long long)t.m * t.n, st, ops, t, kblocks, status);
    if (e != cudaSuccess) return e;
    p.first = i == 0;
    p.words = words;
    p.k = (int)up(words, kPairK);
    p.wm = a.dw ? (int)up(words, kPairTile) : 0;
    p.words_first = p.wk / p.wslices > p.k / (p.slices > 0 ? p.slices : 1);
    e = pair_launch<xent_products_kernel<T>>(
        true, (long long)p.m * p.n * p.slices + (long long)p.wm * p.n * p.wslices, st, p, status);
    if (e == cudaSuccess && a.dw && p.wslices > 1)
      e = add_slices(p.wsums, words * a.dim, p.wslices, unit, static_cast<T *>(a.dw) + t.v0 * a.dim, st);
    if (e != cudaSuccess) return e;
  }
  if (!a.dx || p.dx) return cudaSuccess;
  return add_slices(p.sums, a.tokens * a.dim, p.slices, unit, static_cast<T *>(a.dx), st);
}

}  // namespace

size_t xent_workspace_bytes(int dtype, const XentArgs &a, bool grad) {
  return a.tokens == 0 ? 0 : Layout(dtype, a, grad).bytes + 240;
}

cudaError_t launch_xent(int dtype, const XentArgs &a, void *workspace, cudaStream_t st) {
  char *ws = first_boundary(workspace);
  switch (dtype) {
    case FFT_ELEM_F32: return xent_t<float>(dtype, a, ws, st);
    case FFT_ELEM_BF16: return xent_t<__nv_bfloat16>(dtype, a, ws, st);
    default: return xent_t<__half>(dtype, a, ws, st);
  }
}

cudaError_t launch_xent_grad(int dtype, const XentArgs &a, void *workspace, cudaStream_t st) {
  char *ws = first_boundary(workspace);
  if (a.tokens == 0)
    return a.dw ? cudaMemsetAsync(a.dw, 0, (size_t)a.vocabulary * a.dim * elem_bytes(dtype), st)
                : cudaSuccess;
  switch (dtype) {
    case FFT_ELEM_F32: return xent_grad_t<float>(dtype, a, ws, st);
    case FFT_ELEM_BF16: return xent_grad_t<__nv_bfloat16>(dtype, a, ws, st);
    default: return xent_grad_t<__half>(dtype, a, ws, st);
  }
}

}  // namespace fftgb
