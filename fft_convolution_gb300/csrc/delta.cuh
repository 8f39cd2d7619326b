// delta.cuh -- the gated delta rule over whole sequences, in chunks of 64
// tokens.
//
// Within a chunk write G_i = g_1 + ... + g_i, gamma_i = e^{G_i}, Gamma =
// gamma_64, D_ij = e^{G_i - G_j}, and with the state S0 that enters it
//   A_ij = [j < i] D_ij k_i . k_j,          M_ij = [j <= i] D_ij q_i . k_j,
//   Y = V - gamma K S0,                     E = (I + A beta)^-1 Y,
//   U = beta E,                             O = scale (gamma Q S0 + M U),
//   S1 = Gamma S0 + (K Gamma / gamma)^T U,
// which is the token-by-token recurrence solved for all u_i at once (E_i is
// what the state misses of v_i when token i is read).  Backwards, with dS
// the gradient of S1:
//   dU = scale M^T dO + (K Gamma / gamma) dS,   F = (I + beta A)^-T dU,
//   dV = beta F,                                dbeta_i = E_i . F_i,
//   dS0 = Gamma dS + scale (gamma Q)^T dO - (gamma beta K)^T F,
// and dq, dk, dg from E, F, S0 and dS (delta_grad.cuh).
//
// Decays only ever appear as e^{G_i - G_j} with j <= i, never as a quotient:
// however fast a head forgets, nothing overflows.
//
// Kernels: delta_prep (all chunks in parallel: the triangular inverse and M),
// delta_scan (one block per sequence, head and 128 columns of v walks the
// chunks, the state in registers), and for gradients the same scan backwards in
// the same launch and one more kernel over all chunks.
//
// Precision: products run on the tensor cores in fp16 with fp32
// accumulators.  A row of an operand is first scaled by a power of two that
// brings its largest value to 1 .. 2 (undone on the product's row or column,
// exactly), so fp16's range never matters; and whatever is not exactly fp16
// to begin with (the state, E, U, the inverse, M, fp32 inputs) enters as the
// sum of two fp16 values, of which the products leading x leading, leading x
// trailing and trailing x leading are taken.  22 significand bits count that
// way, at two to three times the products: results in fp32 are about as good
// as fp32 arithmetic's (8192 tokens: the final state 2.3e-7 off, the gradients of
// 16384 tokens 3e-7 to 8e-7, up to 1.9 times the error of elementary fp32
// operations; with pairs of bf16, which need no scaling, a test of 256 tokens was
// 6e-6 off, with single bf16 values 2e-3).  What one scale covers loses digits
// where it is small: in a chunk whose first half reads a state of 2^12 (2^16,
// 2^20) that a decay then drops, results of size 1 are 4e-6 (6e-5, 5e-4) off.
#pragma once

#include "seq.h"
#include "tcgen05.cuh"

namespace fftgb {

constexpr int kChunk = 64;
constexpr float kMinLogDecay = -128.0f;  // e^-128 is 0 in fp32: smaller g change nothing

// One 64 x 64 fp16 tile.
constexpr int kTile = 64 * 128;

// What the scans need of a chunk is laid out by delta_prep as they want it in
// shared memory, in two images.  Per key head the tiles of K and Q, rows
// scaled: for each 64 columns of dk the tile of K, then that of Q; fp32
// inputs: first all leading, then all trailing parts.
__host__ __device__ constexpr int kq_bytes(int dk, int terms) { return terms * 2 * (dk / 64) * kTile; }
// Per value head two 64 x 64 matrices (leading and trailing tile of each),
// rows scaled, eight factors per token, and eight numbers of the chunk: its decay
// Gamma and bounds (delta_prep.cuh).
constexpr int kGates = 8;
constexpr int kChunkAt = kGates * 64;  // in floats, after the tiles
constexpr int kImageBytes = 4 * kTile + kGates * 64 * 4 + 32;

// What the gradients' kernel takes from the scans, per chunk, value head and
// 128 columns of v: the states S0 and dS (DK rows), E, F and dO (64 rows) as
// left and right operands of products over v.  A slab is 16 columns of v, one
// step of the tensor cores: [leading, trailing part][rows / 8][16 columns][8
// rows] of fp16, so a thread of a scan, which owns a column, stores 16 bytes
// and neighbouring lanes neighbouring ones.  One power of two scales a whole
// matrix (products over v admit no scale per column); the inverses are kept.
constexpr int kSlab = 16, kSlabs = 128 / kSlab;
__host__ __device__ constexpr int slab_part(int rows) { return rows * kSlab * 2; }
enum { kScaleS, kScaleE, kScaleD, kScaleF, kScaleO, kScales = 8 };

// Where the chunks of packed sequences lie (device arrays of batch + 1
// entries, both null for sequences of one length).
struct DeltaPlan {
  const int *row0;    // first row of each sequence, made ascending and in range
  const int *chunk0;  // chunks before each sequence
  long long chunks_max;
  int per_seq;  // chunks of each sequence of one length
};

struct DeltaChunk {
  long long b;     // sequence
  long long row;   // first token (of the sequence, or of the packed rows)
  int n;           // tokens, 1 .. 64
};

__device__ __forceinline__ bool delta_chunk(const DeltaArgs &a, const DeltaPlan &p, long long ci,
                                            DeltaChunk &c) {
  if (p.chunk0) {
    if (ci >= p.chunk0[a.batch]) return false;
    long long lo = 0, hi = a.batch - 1;  // the last sequence that starts at or before chunk ci
    while (lo < hi) {
      const long long mid = (lo + hi + 1) >> 1;
      if (p.chunk0[mid] <= ci) lo = mid;
      else hi = mid - 1;
    }
    c.b = lo;
    const int k = (int)(ci - p.chunk0[lo]);
    c.row = (long long)p.row0[lo] + (long long)k * kChunk;
    const long long left = p.row0[lo + 1] - c.row;
    c.n = left < kChunk ? (int)left : kChunk;
  } else {
    c.b = ci / p.per_seq;
    c.row = (ci % p.per_seq) * kChunk;
    const long long left = a.tokens - c.row;
    c.n = left < kChunk ? (int)left : kChunk;
  }
  return c.n > 0;
}

// The parts of a call's workspace, by their offsets in bytes.
struct DeltaLayout {
  long long chunks;        // at most
  size_t row0, chunk0;     // packed: the sequences' first rows and chunks
  size_t kq, images;       // chunks x kheads, chunks x vheads
  size_t back, state, dstate, e, f, o, scales;  // gradients only
  size_t bytes;
  DeltaLayout(const DeltaArgs &a, bool packed, bool grad) {
    chunks = packed ? (a.tokens + (kChunk - 1) * a.batch) / kChunk
                    : a.batch * ((a.tokens + kChunk - 1) / kChunk);
    size_t at = 0;
    auto take = [&](size_t n) {
      const size_t here = at;
      at += (n + 255) & ~(size_t)255;
      return here;
    };
    const size_t ch = (size_t)chunks * a.vheads, chv = ch * ((a.dv + 127) / 128);
    const int dk = a.dk <= 64 ? 64 : 128;
    row0 = take(packed ? (a.batch + 1) * sizeof(int) : 0);
    chunk0 = take(packed ? (a.batch + 1) * sizeof(int) : 0);
    kq = take((size_t)chunks * a.kheads * kq_bytes(dk, a.terms));
    images = take(ch * kImageBytes);
    back = take(grad ? ch * kImageBytes : 0);
    state = take(grad ? chv * 128 * dk * 4 : 0);
    dstate = take(grad ? chv * 128 * dk * 4 : 0);
    e = take(grad ? chv * 64 * 128 * 4 : 0);
    f = take(grad ? chv * 64 * 128 * 4 : 0);
    o = take(grad ? chv * 64 * 128 * 2 * a.terms : 0);
    scales = take(grad ? chv * kScales * 4 : 0);
    bytes = at;
  }
};

// Elements [token][*] of a head's rows.
template <typename T>
__device__ __forceinline__ const T *head_rows(const void *p, const DeltaStride &s, long long b,
                                              long long row, long long head) {
  return static_cast<const T *>(p) + b * s.seq + row * s.tok + head * s.head;
}

// fp16 values per input element: one holds bf16 and fp16 elements of a scaled
// row, fp32 takes two.
template <typename T> struct Terms { static constexpr int value = 1; };
template <> struct Terms<float> { static constexpr int value = 2; };

// Eight elements of a row; zero from `left` elements on.
template <typename T> struct Row8 {
  static constexpr int N = sizeof(T) / 2;  // 16-byte words
  uint4 raw[N];
  __device__ __forceinline__ void load(const T *p, int left, bool vec) {
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = make_uint4(0, 0, 0, 0);
    if (left <= 0) return;
    if (vec && left >= 8) {
#pragma unroll
      for (int i = 0; i < N; ++i) raw[i] = reinterpret_cast<const uint4 *>(p)[i];
    } else {
      T *t = reinterpret_cast<T *>(raw);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) t[i] = p[i];
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const T *t = reinterpret_cast<const T *>(raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_acc(t[i]);
  }
};

__device__ __forceinline__ float max8(const float (&f)[8]) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  return m;
}
// Largest value over aligned groups of W lanes.
template <int W> __device__ __forceinline__ float lane_max(float m) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

__device__ __forceinline__ void split8(const float (&f)[8], float s, uint4 &hi, uint4 &lo) {
  split2(mul2(make_float2(f[0], f[1]), both(s)), hi.x, lo.x);
  split2(mul2(make_float2(f[2], f[3]), both(s)), hi.y, lo.y);
  split2(mul2(make_float2(f[4], f[5]), both(s)), hi.z, lo.z);
  split2(mul2(make_float2(f[6], f[7]), both(s)), hi.w, lo.w);
}
// Byte offset of the 16-byte piece c (8 columns) of row r in a row of tiles
// `tile` bytes apart.
__device__ __forceinline__ int piece_at(int r, int c, int tile) {
  return (c >> 3) * tile + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Whether 16-byte loads fit every row of a head.
template <typename T>
__host__ __device__ __forceinline__ bool vec_rows(const void *p, const DeltaStride &s) {
  return ((uintptr_t)p & 15u) == 0 && (s.seq * sizeof(T)) % 16 == 0 &&
         (s.tok * sizeof(T)) % 16 == 0 && (s.head * sizeof(T)) % 16 == 0;
}

// A wait that also ends when another warp has given up; `failed` is a word
// in shared memory, `status` the device status word.
__device__ __forceinline__ bool wait_or_fail(uint64_t *bar, uint32_t parity, volatile int *failed,
                                             int *status) {
  if (bar_poll(bar, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t it = 0; it < (1u << 24); ++it) {
    if (bar_poll(bar, parity)) return true;
    if (*failed || clock64() - t0 > 8000000000ll) break;  // about 4 s
  }
  *failed = 1;
  atomicExch(status, 1);  // kDeviceErrorTimeout
  return false;
}

}  // namespace fftgb
