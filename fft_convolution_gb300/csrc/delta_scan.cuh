// delta_scan.cuh -- the gated delta rule from chunk to chunk (delta.cuh).
//
// One block walks a sequence's chunks for one head and 128 columns of v, with
// everything transposed: a column of v is a lane of tensor memory and a row
// of the left operands, K and Q in shared memory serve as right operands as
// they come (K-major for S^T K^T, MN-major for U^T K).  Per chunk
//   P = S^T K^T, N = S^T Q^T;  Y = V^T - P gamma;  E = Y T^T (T the inverse);
//   U = E beta;  W = U Gamma / gamma;  S^T <- S^T Gamma + W K;
//   O^T = scale (N gamma + U M^T).
// Four threads own a column of v, each with a quarter of the tokens and of
// the state's columns: the state itself stays in their registers in fp32,
// and what they hand to the tensor cores (S, Y, U, W) is scaled by a power of
// two and split into two fp16 values.  Only P -> Y -> E -> U -> S is a chain;
// N, U M^T, the output and all loads run beside it.  (Both products of the
// output keep their own scales and meet in fp32: one may be far below the
// other.)  So the scales do not come from the values (finding the largest of a
// column takes the four threads a barrier at each step of the chain) but from
// bounds on them: from the largest values of V and of the state, which are found
// beside the chain, and the chunk's bounds.  The scale brings the bound to 2^14;
// values down to 2^-16 of the bound keep all their digits.  A bound counts as
// kApart of what it is computed from at least: the quotient of two scales stays
// finite then (a chunk that writes nothing has a bound of 0 on U and W, however
// large the state).
//
// The chain bounds it: a chunk takes 4900 clocks, of which the tensor cores work
// about 1400; the rest are four trips from them through registers and back, with
// 65% of the issue slots used.  8192 tokens of 32 heads of 128 x 128 (32 blocks,
// 128 chunks each) take 333 us; HBM is idle meanwhile.  16-bit rows on 16-byte
// boundaries (STAGED) leave the 96 registers of a thread enough for that.
// Others, all of fp32 among them, spill up to 94 bytes; where both scans of the
// gradients share a kernel (delta_back.cuh) heads of 128 spill 4, not staged 126
// to 250.
//
// Roles: 16 warps of arithmetic (two per scheduler left its issue slots 60%
// empty), one thread that issues the products, a warp that fetches the chunks'
// images ahead (bulk copies) and two that store.
//
// Tensor memory (512 columns):
//   W K (fp32)       0 .. DK - 1
//   S (two fp16)     128, 192        P, then E     256 .. 319
//   Y, then U        320, 352        W, then U M^T  384, 416
//   N                448 .. 511
#pragma once

#include "delta.cuh"

namespace fftgb {

constexpr int kScanWarps = 16;                       // of arithmetic
constexpr int kScanGroups = kScanWarps / 4;          // threads that share a column of v
constexpr int kScanTok = 64 / kScanGroups;           // tokens of each
constexpr int kScanThreads = (kScanWarps + 4) * 32;
constexpr int kScanStages = 2;
constexpr float kApart = 0x1p-86f;

// 64 tokens x 128 columns of a 16-bit type.
constexpr int kRows16 = 64 * 128 * 2;
// Stage: the tiles of K and Q, the head's image up to its factors, and
// (STAGED) the rows of V (backwards: of dO); 1024-byte aligned.
__host__ __device__ constexpr int scan_stage_bytes(int dk, int terms, bool staged) {
  return kq_bytes(dk, terms) + 4 * kTile + (staged ? kRows16 : 0);
}
// Two stages, (STAGED) the rows of O (of dV) on their way out, and the factors
// of four chunks: a chunk's output is still scaled while the stage of its
// tiles is being filled again.
constexpr int kGateBytes = kImageBytes - 4 * kTile, kGateRing = 4;
__host__ __device__ constexpr size_t scan_smem(int dk, int terms, bool staged) {
  return 1024 + (size_t)kScanStages * scan_stage_bytes(dk, terms, staged) +
         (staged ? kRows16 : 0) + kGateRing * kGateBytes;
}

struct ScanBars {
  uint64_t full[kScanStages], empty[kScanStages];
  uint64_t p, n, e, s, o;       // products done: P, X (backwards), E, W K, N and U M^T
  uint64_t y, w, u, sb, of;     // operands ready: Y, W, U, S; N and U M^T read
  uint64_t put, got;            // STAGED: rows of O in shared memory; copied out
  uint64_t done;                // every product
};

// The chunks of one sequence.
struct ScanSpan {
  long long b, row0, chunk0;
  long long rows;
  int chunks;
};
__device__ __forceinline__ ScanSpan scan_span(const DeltaArgs &a, const DeltaPlan &p, long long b) {
  ScanSpan s;
  s.b = b;
  if (p.chunk0) {
    s.row0 = p.row0[b];
    s.rows = p.row0[b + 1] - s.row0;
    s.chunk0 = p.chunk0[b];
    s.chunks = p.chunk0[b + 1] - p.chunk0[b];
  } else {
    s.row0 = 0;
    s.rows = a.tokens;
    s.chunk0 = b * p.per_seq;
    s.chunks = p.per_seq;
  }
  return s;
}

// Row of a contiguous [sequence][token][head][dv] array.
__device__ __forceinline__ long long out_row(const DeltaArgs &a, long long b, long long row,
                                             bool packed, int h) {
  return ((packed ? row : b * a.tokens + row) * a.vheads + h) * a.dv;
}

// The loading warp: the chunks' images into the stages and, STAGED, the rows
// x of v's type (128 columns from column c0; where the chunk has fewer than 64
// tokens its last row again: its values meet factors of 0, which only
// finite ones leave 0).  The rows go by 16-byte copies: as one bulk copy per
// row of 256 bytes they took longer than the rest of the chunk's work.
template <typename T, int DK, bool STAGED>
__device__ __forceinline__ void scan_load(const DeltaArgs &a, const ScanSpan &sp, int h,
                                          bool backwards, const char *kq, const char *images,
                                          const T *x, long long step, int c0, char *stages,
                                          char *ring, ScanBars *bars, volatile int *failed,
                                          int *status, int lane) {
  constexpr int NT = Terms<T>::value, ST = kScanStages;
  constexpr int kStage = scan_stage_bytes(DK, NT, STAGED);
  const int hk = h / (a.vheads / a.kheads);
  const int pieces = (a.dv - c0 < 128 ? a.dv - c0 : 128) / 8;
  int issued = 0;
  for (int it = 0; it < sp.chunks; ++it) {
    const int ci = backwards ? sp.chunks - 1 - it : it;
    const long long c = sp.chunk0 + ci;
    const int s = it % ST;
    const bool ok = it < ST || wait_or_fail(&bars->empty[s], (it / ST - 1) & 1, failed, status);
    if (!__all_sync(0xffffffffu, ok)) break;
    char *stage = stages + s * kStage;
    if (lane == 0) {
      const char *image = images + (c * a.vheads + h) * (long long)kImageBytes;
      bar_arrive_tx(&bars->full[s], kq_bytes(DK, NT) + kImageBytes);
      bulk_load(stage, kq + (c * a.kheads + hk) * (long long)kq_bytes(DK, NT), kq_bytes(DK, NT),
                &bars->full[s]);
      bulk_load(stage + kq_bytes(DK, NT), image, 4 * kTile, &bars->full[s]);
      bulk_load(ring + (it % kGateRing) * kGateBytes, image + 4 * kTile, kGateBytes,
                &bars->full[s]);
    }
    if constexpr (STAGED) {
      const long long r0 = (long long)ci * kChunk;
      const int last = (int)(sp.rows - r0 < kChunk ? sp.rows - r0 : kChunk) - 1;
      const uint32_t dst = smem_u32(stage + kStage - kRows16) + (lane & 15) * 16;
      const T *src = x + r0 * step + (lane & 15) * 8;
      if ((lane & 15) < pieces) {
#pragma unroll 16
        for (int r = lane >> 4; r < kChunk; r += 2)
          copy16(dst + r * 256, src + (r < last ? r : last) * step);
      }
      copy_arrive(&bars->full[s]);
    }
    issued = it + 1;
  }
  // Given up: no copy may land after the block has gone.
  if (*failed) {
    copy_wait_all();
    for (int it = issued > ST ? issued - ST : 0; it < issued; ++it)
      bar_wait(&bars->full[it % ST], (it / ST) & 1);
  }
}

// A thread's values of one column of v, 16 tokens.  Into the rows in shared
// memory two lanes put their columns' values of a token in one word each, one
// lane the even tokens, the other the odd ones (stores of two bytes took four
// times as long); odd rows have their 64-byte halves exchanged, so that the
// two lanes' words lie in different banks.
template <typename T> struct TokenValues {
  T v[kScanTok];
  __device__ __forceinline__ void set(int j, float2 x) {
    v[2 * j] = from_acc<T>(x.x);
    v[2 * j + 1] = from_acc<T>(x.y);
  }
  __device__ __forceinline__ T get(int j) const { return v[j]; }
  __device__ __forceinline__ void put(char *, int, int, int) const {}  // not staged
};
template <typename T> struct TokenPairs {
  uint32_t w[kScanTok / 2];
  __device__ __forceinline__ T get(int j) const {
    const uint16_t x = (uint16_t)(j & 1 ? w[j / 2] >> 16 : w[j / 2]);
    return *reinterpret_cast<const T *>(&x);
  }
  __device__ __forceinline__ void put(char *rows, int tok, int col, int lane) const {
    const int odd = lane & 1;
    char *at = rows + (tok + odd) * 256 + (((col & ~1) * 2) ^ (odd << 6));
#pragma unroll
    for (int j = 0; j < kScanTok / 2; ++j) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, w[j], 1);
      const uint32_t x = odd ? __byte_perm(o, w[j], 0x7632) : __byte_perm(w[j], o, 0x5410);
      *reinterpret_cast<uint32_t *>(at + j * 512) = x;
    }
  }
};
template <> struct TokenValues<__nv_bfloat16> : TokenPairs<__nv_bfloat16> {
  __device__ __forceinline__ void set(int j, float2 x) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x.x, x.y);
    w[j] = *reinterpret_cast<const uint32_t *>(&p);
  }
};
template <> struct TokenValues<__half> : TokenPairs<__half> {
  __device__ __forceinline__ void set(int j, float2 x) {
    const __half2 p = __floats2half2_rn(x.x, x.y);
    w[j] = *reinterpret_cast<const uint32_t *>(&p);
  }
};

// The two storing warps, STAGED: the chunks' rows from shared memory to the
// contiguous array [sequence][token][head][dv].  `which`: half of the rows.
template <typename T>
__device__ __forceinline__ void scan_store(const DeltaArgs &a, const ScanSpan &sp, bool packed,
                                           int h, bool backwards, void *out, int c0,
                                           const char *rows, ScanBars *bars,
                                           volatile int *failed, int *status, int which,
                                           int lane) {
  const int pieces = (a.dv - c0 < 128 ? a.dv - c0 : 128) / 8;
  const long long step = (long long)a.vheads * a.dv;
  for (int it = 0; it < sp.chunks; ++it) {
    const int ci = backwards ? sp.chunks - 1 - it : it;
    const bool ok = wait_or_fail(&bars->put, it & 1, failed, status);
    if (!__all_sync(0xffffffffu, ok)) break;
    const long long row = (long long)ci * kChunk;
    const int n = (int)(sp.rows - row < kChunk ? sp.rows - row : kChunk);
    T *dst = static_cast<T *>(out) + out_row(a, sp.b, sp.row0 + row, packed, h) + c0 +
             (lane & 15) * 8;
    const char *src = rows + (((lane & 15) * 16) ^ ((lane >> 4) << 6));
    if ((lane & 15) < pieces) {
      const int r0 = which * 32 + (lane >> 4);
#pragma unroll
      for (int b = 0; b < 32; b += 16) {
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          x[k] = *reinterpret_cast<const uint4 *>(src + (r0 + b + 2 * k) * 256);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (r0 + b + 2 * k < n) *reinterpret_cast<uint4 *>(dst + (r0 + b + 2 * k) * step) = x[k];
      }
    }
    __syncwarp();
    if (lane == 0) bar_arrive(&bars->got);
  }
}

constexpr uint32_t idesc_tokens = mma_desc(128, 64, false, false);

// Products of trailing parts come first: the accumulator cuts off below its
// last bit at every step, which costs little while it is small (dbeta of 16384
// tokens: 7.7e-7 off, with the leading parts first 1.9e-6).

// S^T X^T into `d` (64 columns): left operand the state's two parts, right
// one the chunk's X (K or Q).
template <int DK, int NT>
__device__ __forceinline__ void mma_state(uint32_t d, uint32_t hi, uint32_t lo, uint32_t x) {
  constexpr uint32_t kPlane = 2 * (DK / 64) * kTile;
#pragma unroll
  for (int term = NT == 1 ? 1 : 2; term >= 0; --term) {
    const uint32_t ta = term == 1 ? lo : hi, tb = x + (term == 2 ? kPlane : 0);
#pragma unroll
    for (int k = 0; k < DK / 16; ++k)
      mma_ts(d, ta + 8 * k, tile_desc(tb + (k >> 2) * 2 * kTile + (k & 3) * 32, 16),
             idesc_tokens, term < (NT == 1 ? 1 : 2) || k > 0);
  }
}
// A B^T for 64-token A (two parts; ONE: the leading one is all of it) and a
// 64 x 64 matrix of the image.
template <bool ONE = false>
__device__ __forceinline__ void mma_inner(uint32_t d, uint32_t hi, uint32_t lo, uint32_t m,
                                          bool accumulate) {
#pragma unroll
  for (int term = 2; term >= 0; --term) {
    if (ONE && term == 1) continue;
    const uint32_t ta = term == 1 ? lo : hi, tb = m + (term == 2 ? kTile : 0);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      mma_ts(d, ta + 8 * k, tile_desc(tb + k * 32, 16), idesc_tokens,
             accumulate || term < 2 || k > 0);
  }
}
// A X for 64-token A and the chunk's X (K or Q) as 64 tokens x DK.
template <int DK, int NT>
__device__ __forceinline__ void mma_update(uint32_t d, uint32_t hi, uint32_t lo, uint32_t x,
                                           bool accumulate) {
  constexpr uint32_t idesc = mma_desc(128, DK, false, true);
  constexpr uint32_t kPlane = 2 * (DK / 64) * kTile;
#pragma unroll
  for (int term = NT == 1 ? 1 : 2; term >= 0; --term) {
    const uint32_t ta = term == 1 ? lo : hi, tb = x + (term == 2 ? kPlane : 0);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      mma_ts(d, ta + 8 * k, tile_desc(tb + k * 2048, 2 * kTile), idesc,
             accumulate || term < (NT == 1 ? 1 : 2) || k > 0);
  }
}

// 16 scaled values to the two parts of a left operand (8 packed columns each).
__device__ __forceinline__ void put_split(uint32_t hi_at, uint32_t lo_at, const float2 (&f)[8]) {
  uint32_t hi[8], lo[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) split2(f[j], hi[j], lo[j]);
  tmem_st(hi_at, hi);
  tmem_st(lo_at, lo);
}
// The leading part alone.
__device__ __forceinline__ void put_lead(uint32_t at, const float2 (&f)[8]) {
  uint32_t hi[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const __half2 h = __float22half2_rn(f[j]);
    hi[j] = *reinterpret_cast<const uint32_t *>(&h);
  }
  tmem_st(at, hi);
}
__device__ __forceinline__ float max16(float m, const float2 (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(f[j].x), fabsf(f[j].y)));
  return m;
}
template <int N> __device__ __forceinline__ float2 pair(const uint32_t (&r)[N], int j) {
  return make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
}
// Factors of tokens 2j, 2j + 1 of a thread's.
__device__ __forceinline__ float2 gate(const float *g, int j) {
  return *reinterpret_cast<const float2 *>(g + 2 * j);
}

// One arrival per warp, after every lane's accesses to tensor memory.
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) bar_arrive(bar);
}

// 16 scaled values of a thread's column, rows m .. m + 15, to the slabs of a
// matrix of `rows` rows; TWO: both parts, else the leading one.
template <bool TWO>
__device__ __forceinline__ void put_slab(char *matrix, int rows, int parts, int m, int col,
                                         const float2 (&f)[8], bool live) {
  char *at = matrix + (col >> 4) * (parts * slab_part(rows)) + (m >> 3) * 256 + (col & 15) * 16;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      split2(f[4 * p + j], hi[j], lo[j]);
      if (!live) hi[j] = lo[j] = 0;
    }
    *reinterpret_cast<uint4 *>(at + p * 256) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if constexpr (TWO)
      *reinterpret_cast<uint4 *>(at + p * 256 + slab_part(rows)) =
          make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// Bounds over all 128 columns of v, for the scales of what is kept for the
// gradients: every warp enters its own before it hands over an operand, and
// reads the block's once the product that waited for all of them is there.
// Four chunks' entries; those of the chunk after next are cleared.
constexpr int kTops = 3;
struct BlockBounds {
  unsigned top[4][kTops];
  __device__ __forceinline__ void enter(int it, int which, float b, int lane) {
    // (of values that are not negative the bits are in order)
    const unsigned m = __reduce_max_sync(0xffffffffu, __float_as_uint(b));
    if (lane == 0) atomicMax(&top[it & 3][which], m);
  }
  __device__ __forceinline__ float scale(int it, int which) const {
    return bound_scale(__uint_as_float(*(volatile const unsigned *)&top[it & 3][which]));
  }
  __device__ __forceinline__ void clear(int it) {
    for (int k = 0; k < kTops; ++k) top[(it + 2) & 3][k] = 0;
  }
};

// The largest of what the four threads of a column of v bring, twice.  Their
// four warps meet at a barrier of their own; the two halves of `box` alternate,
// so one barrier per agreement is enough.
struct RowAgree {
  float2 (*box)[kScanGroups][128];
  int row, group, quarter, turn;
  __device__ __forceinline__ float2 largest(float a, float b) {
    box[turn][group][row] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(1 + quarter), "n"(kScanGroups * 32) : "memory");
#pragma unroll
    for (int g = 0; g < kScanGroups; ++g) {
      const float2 o = box[turn][g][row];
      a = fmaxf(a, o.x);
      b = fmaxf(b, o.y);
    }
    turn ^= 1;
    return make_float2(a, b);
  }
};

constexpr uint32_t kColD = 0, kColSh = 128, kColSl = 192, kColP = 256, kColYh = 320, kColYl = 352,
                   kColWh = 384, kColWl = 416, kColN = 448, kColUM = kColWh;

// Barriers and tensor memory of a scan: returns the base column.
__device__ __forceinline__ uint32_t scan_begin(ScanBars &bars, uint32_t *slot, volatile int *failed,
                                               bool staged, int tid, int warp) {
  if (warp == kScanWarps) tmem_alloc(slot, 512);
  if (tid == 0) {
    for (int s = 0; s < kScanStages; ++s) {
      bar_init(&bars.full[s], staged ? 33 : 1);
      bar_init(&bars.empty[s], 1 + kScanWarps);
    }
    for (uint64_t *b : {&bars.p, &bars.n, &bars.e, &bars.s, &bars.o, &bars.done}) bar_init(b, 1);
    bar_init(&bars.got, 2);
    for (uint64_t *b : {&bars.y, &bars.w, &bars.u, &bars.sb, &bars.of, &bars.put})
      bar_init(b, kScanWarps);
    *failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return __shfl_sync(0xffffffffu, *slot, 0);
}

// SAVE leaves for the gradients the state that entered each chunk and E, as
// slabs (delta.cuh).
// STAGED: V comes and O goes through shared memory by bulk copies of rows
// (16-bit types on 16-byte boundaries); else straight from and to HBM.
template <typename T, int DK, bool SAVE, bool STAGED>
__device__ __forceinline__ void delta_scan(const DeltaArgs &a, const DeltaPlan &plan, unsigned block,
                                           const char *kq, const char *images, char *states,
                                           char *es, float *scales, int *status) {
  extern __shared__ char smem_raw[];
  __shared__ ScanBars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int failed;
  __shared__ float2 box[2][kScanGroups][128];
  __shared__ BlockBounds bounds;
  constexpr int NT = Terms<T>::value, ST = kScanStages;
  constexpr int kStage = scan_stage_bytes(DK, NT, STAGED);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int blocks_v = (a.dv + 127) / 128;
  const int vb = block % blocks_v;
  const int h = (block / blocks_v) % a.vheads;
  const ScanSpan sp = scan_span(a, plan, block / blocks_v / a.vheads);
  char *stages = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  if (SAVE && tid < 4 * kTops) bounds.top[tid / kTops][tid % kTops] = 0;
  const uint32_t tm = scan_begin(bars, &tmem_slot, &failed, STAGED, tid, warp);
  char *ring = stages + ST * kStage + (STAGED ? kRows16 : 0);
  auto wait = [&](uint64_t *b, uint32_t parity) { return wait_or_fail(b, parity, &failed, status); };

  if (warp >= kScanWarps + 2) {
    if constexpr (STAGED)
      if (a.o)
        scan_store<T>(a, sp, plan.chunk0 != nullptr, h, false, a.o, vb * 128, stages + ST * kStage,
                      &bars, &failed, status, warp - kScanWarps - 2, lane);
  } else if (warp == kScanWarps + 1) {
    scan_load<T, DK, STAGED>(a, sp, h, false, kq, images,
                             head_rows<T>(a.v, a.sv, sp.b, sp.row0, h) + vb * 128, a.sv.tok,
                             vb * 128, stages, ring, &bars, &failed, status, lane);
  } else if (warp == kScanWarps) {
    // The whole warp walks along, one lane issues.
    for (int it = 0; it < sp.chunks; ++it) {
      const int s = it % ST;
      const uint32_t ph = it & 1;
      const uint32_t k = smem_u32(stages) + s * kStage;
      const uint32_t q = k + kTile, image = k + kq_bytes(DK, NT);
      if (!wait(&bars.full[s], (it / ST) & 1) || !wait(&bars.sb, ph)) break;
      tc_fence_after();
      if (elect_one()) {
        mma_state<DK, NT>(tm + kColP, tm + kColSh, tm + kColSl, k);
        mma_commit(&bars.p);
      }
      __syncwarp();
      if (!wait(&bars.y, ph)) break;
      tc_fence_after();
      if (elect_one()) mma_inner<>(tm + kColP, tm + kColYh, tm + kColYl, image, false);
      __syncwarp();
      // E is told of when U M^T has been read too: W will lie there.
      if (it > 0 && !wait(&bars.of, ph ^ 1)) break;
      tc_fence_after();
      if (elect_one()) {
        mma_commit(&bars.e);
        mma_state<DK, NT>(tm + kColN, tm + kColSh, tm + kColSl, q);
        mma_commit(&bars.n);
      }
      __syncwarp();
      if (!wait(&bars.w, ph)) break;
      tc_fence_after();
      if (elect_one()) {
        mma_update<DK, NT>(tm + kColD, tm + kColWh, tm + kColWl, k, false);
        mma_commit(&bars.s);
      }
      __syncwarp();
      if (!wait(&bars.u, ph) || !wait(&bars.s, ph)) break;  // (W has been used)
      tc_fence_after();
      if (elect_one()) {
        mma_inner<>(tm + kColUM, tm + kColYh, tm + kColYl, image + 2 * kTile, false);
        mma_commit(&bars.o);
        mma_commit(&bars.empty[s]);
      }
      __syncwarp();
    }
    if (elect_one()) {
      mma_commit(&bars.done);
      bar_wait(&bars.done, 0);
    }
    __syncwarp();
  } else {
    const int group = warp >> 2;             // its tokens and state columns
    const int row = (warp & 3) * 32 + lane;  // column of v within the block
    const uint32_t lb = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const int dvr = vb * 128 + row;
    const bool live = dvr < a.dv;
    constexpr int TK = kScanTok, SC = DK / kScanGroups, SP = SC / 16;  // state columns in parts of 16
    const long long sat = ((sp.b * a.vheads + h) * a.dk) * (long long)a.dv + dvr;
    RowAgree agree{box, row, group, warp & 3, 0};
    auto saved = [&](long long c) { return ((sp.chunk0 + c) * a.vheads + h) * blocks_v + vb; };
    auto gates_of = [&](int it) {
      return reinterpret_cast<const float *>(ring + (it % kGateRing) * kGateBytes);
    };
    // V of a chunk, fetched while the chunk before is worked on: every load is
    // unconditional (of the last row and column where there is none) and its
    // value not looked at before it is needed, so all are under way at once.
    T vr[STAGED ? 1 : TK];
    const T *vcol = head_rows<T>(a.v, a.sv, sp.b, sp.row0, h) + (live ? dvr : a.dv - 1);
    auto fetch_v = [&](int c) {
      if constexpr (!STAGED) {
        const long long r0 = (long long)c * kChunk;
        const int last = (int)(sp.rows - r0 < kChunk ? sp.rows - r0 : kChunk) - 1;
        const T *v = vcol + r0 * a.sv.tok;
#pragma unroll
        for (int j = 0; j < TK; ++j) {
          const int t = group * TK + j < last ? group * TK + j : last;
          vr[j] = v[(long long)t * a.sv.tok];
        }
      }
    };
    // The state times ss, its scale as an operand: ss changes from chunk to
    // chunk, the values' rounding does not.
    float2 S[SP][8];
    float ss = 1.0f;
    auto put_state = [&](long long c) {
#pragma unroll
      for (int p = 0; p < SP; ++p) {
        const int col = group * SC + p * 16;
        put_split(lb + kColSh + col / 2, lb + kColSl + col / 2, S[p]);
      }
      tmem_wait_st();
      warp_arrive(&bars.sb, lane);
      if constexpr (SAVE) {
        const float xs = bounds.scale(c - 1, 1), by = scale_inverse(ss) * xs;
#pragma unroll
        for (int p = 0; p < SP; ++p) {
          float2 f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = mul2(S[p][j], both(by));
          put_slab<true>(states + saved(c) * (512 * DK), DK, 2, group * SC + p * 16, row, f, live);
        }
        if (tid == 0) scales[saved(c) * kScales + kScaleS] = scale_inverse(xs);
      }
    };
    auto state_max = [&]() {
      float m = 0.0f;
#pragma unroll
      for (int p = 0; p < SP; ++p) m = max16(m, S[p]);
      return m;
    };
    auto initial = [&](int col) {
      return a.state_in && live && col < a.dk ? a.state_in[sat + (long long)col * a.dv] : 0.0f;
    };
#pragma unroll
    for (int p = 0; p < SP; ++p)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = group * SC + p * 16 + 2 * j;
        S[p][j] = make_float2(initial(col), initial(col + 1));
      }
    // V of chunk c into f, and the largest of it.
    float vmax = 0.0f;
    auto take_v = [&](int c, float2 (&f)[8]) {
      const int s = c % ST;
      if (!wait(&bars.full[s], (c / ST) & 1)) return false;
      const T *vs = reinterpret_cast<const T *>(stages + s * kStage + kStage - kRows16) +
                    group * TK * 128 + row;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f[j] = STAGED ? make_float2(to_acc(vs[2 * j * 128]), to_acc(vs[(2 * j + 1) * 128]))
                      : make_float2(to_acc(vr[STAGED ? 0 : 2 * j]),
                                    to_acc(vr[STAGED ? 0 : 2 * j + 1]));
      vmax = max16(0.0f, f);
      return true;
    };
    // The output of chunk c, whose U had this scale.
    auto put_output = [&](int c, float inv_u) {
      const float *gates = gates_of(c) + group * TK;
      if (!wait(&bars.o, c & 1)) return false;
      if (STAGED && a.o && c > 0 && !wait(&bars.got, (c & 1) ^ 1)) return false;
      tc_fence_after();
      tmem_wait_st();  // (N)
      TokenValues<T> out;
#pragma unroll
      for (int p = 0; p < 2; ++p) {  // (all 16 tokens' at once spill)
        uint32_t r[8], n[8];
        tmem_ld(lb + kColUM + group * TK + 8 * p, r);
        tmem_ld(lb + kColN + group * TK + 8 * p, n);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          out.set(4 * p + j, fma2(pair(r, j), mul2(gate(gates + 4 * 64, 4 * p + j), both(inv_u)),
                                  pair(n, j)));
      }
      warp_arrive(&bars.of, lane);
      if (STAGED && a.o) {
        out.put(stages + ST * kStage, group * TK, row, lane);
      } else if (a.o && live) {
        const long long r0 = sp.row0 + (long long)c * kChunk + group * TK;
        const long long left = sp.rows - (long long)c * kChunk - group * TK;
        T *o = static_cast<T *>(a.o) + out_row(a, sp.b, r0, plan.chunk0 != nullptr, h) + dvr;
        const long long step = (long long)a.vheads * a.dv;
#pragma unroll
        for (int j = 0; j < TK; ++j)
          if (j < left) o[j * step] = out.get(j);
      }
      __syncwarp();
      if (STAGED && lane == 0) bar_arrive(&bars.put);
      return true;
    };
    bool ok = true;
    if (sp.chunks > 0) {
      fetch_v(0);
      const float smax = agree.largest(state_max(), 0.0f).x;
      ss = bound_scale(smax);
      if constexpr (SAVE) {
        bounds.enter(-1, 1, live ? smax : 0.0f, lane);
        asm volatile("bar.sync 5, %0;" ::"n"(kScanWarps * 32) : "memory");
      }
#pragma unroll
      for (int p = 0; p < SP; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) S[p][j] = mul2(S[p][j], both(ss));
      put_state(0);
    }
    float inv_u = 1.0f;  // of the chunk before
    for (int it = 0; it < sp.chunks && ok; ++it) {
      const uint32_t ph = it & 1;
      const float *gates = gates_of(it) + group * TK;
      uint32_t r[16];
      // While P is computed: V, and the scales.
      float2 f[8];
      if (!(ok = take_v(it, f))) break;
      const float2 most = agree.largest(state_max(), vmax);
      const float *chunk = gates_of(it) + kChunkAt;
      const float Gamma = chunk[0], inv_s = scale_inverse(ss), smax = most.x * inv_s;
      const float bw = fmaf(chunk[6], smax, chunk[3] * most.y);
      const float yb = fmaxf(fmaf(chunk[1], smax, most.y), smax * kApart), least = yb * kApart;
      const float ys = bound_scale(yb);
      const float us = bound_scale(
          fmaxf(fmaf(chunk[5], smax, chunk[2] * most.y), least * fmaxf(1.0f, chunk[2])));
      const float wsc = bound_scale(fmaxf(bw, least * fmaxf(1.0f, chunk[3])));
      const float inv_y = scale_inverse(ys);
      const float bs = fmaf(Gamma, smax, 128.0f * bw), next_ss = bound_scale(bs);
      if constexpr (SAVE) {
        bounds.enter(it, 0, live ? fmaxf(fmaf(chunk[7], smax, chunk[4] * most.y), least) : 0.0f, lane);
        bounds.enter(it, 1, live ? bs : 0.0f, lane);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = mul2(f[j], both(ys));
      // Y = V^T - P gamma
      if (!(ok = wait(&bars.p, ph))) break;
      tc_fence_after();
      tmem_ld(lb + kColP + group * TK, r);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f[j] = fma2(mul2(gate(gates, j), both(inv_s * ys)), pair(r, j), f[j]);
      put_split(lb + kColYh + group * 8, lb + kColYl + group * 8, f);
      tmem_wait_st();
      warp_arrive(&bars.y, lane);
      if (lane == 0) bar_arrive(&bars.empty[it % ST]);  // V has been used
      // While E is computed: the output of the chunk before.
      if (it > 0 && !(ok = put_output(it - 1, inv_u))) break;
      inv_u = scale_inverse(us);
      // W = E beta Gamma / gamma, on which the new state waits, then U = E beta
      // (E taken from tensor memory once more, which saves registers).
      if (!(ok = wait(&bars.e, ph))) break;
      tc_fence_after();
      tmem_ld(lb + kColP + group * TK, r);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f[j] = mul2(pair(r, j), mul2(gate(gates + 64, j), both(inv_y * wsc)));
      put_split(lb + kColWh + group * 8, lb + kColWl + group * 8, f);
      tmem_wait_st();
      warp_arrive(&bars.w, lane);
      tmem_ld(lb + kColP + group * TK, r);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f[j] = mul2(pair(r, j), mul2(gate(gates + 2 * 64, j), both(inv_y * us)));
      put_split(lb + kColYh + group * 8, lb + kColYl + group * 8, f);
      if constexpr (SAVE) {
        const float es_scale = bounds.scale(it, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          f[j] = mul2(pair(r, j), mul2(gate(gates + 5 * 64, j), both(inv_y * es_scale)));
        put_slab<true>(es + saved(it) * (64 * 128 * 4), 64, 2, group * TK, row, f, live);
        if (tid == 0) {
          scales[saved(it) * kScales + kScaleE] = scale_inverse(es_scale);
          bounds.clear(it);
        }
      }
      tmem_wait_st();
      warp_arrive(&bars.u, lane);
      // While the new state is computed: N in the output's units.
      if (!(ok = wait(&bars.n, ph))) break;
      tc_fence_after();
      tmem_ld(lb + kColN + group * TK, r);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 n = mul2(pair(r, j), mul2(gate(gates + 3 * 64, j), both(inv_s)));
        r[2 * j] = __float_as_uint(n.x);
        r[2 * j + 1] = __float_as_uint(n.y);
      }
      tmem_st(lb + kColN + group * TK, r);
      const bool more = it + 1 < sp.chunks;
      if (more) fetch_v(it + 1);
      // The new state
      const float keep = Gamma * inv_s * next_ss, add = scale_inverse(wsc) * next_ss;
      if (!(ok = wait(&bars.s, ph))) break;
      tc_fence_after();
#pragma unroll
      for (int p = 0; p < SP; ++p) {
        tmem_ld(lb + kColD + group * SC + p * 16, r);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          S[p][j] = fma2(S[p][j], both(keep), mul2(pair(r, j), both(add)));
      }
      ss = next_ss;
      if (more) put_state(it + 1);
    }
    if (ok && sp.chunks > 0) ok = put_output(sp.chunks - 1, inv_u);
    if (ok && a.state_out && live) {
#pragma unroll
      for (int p = 0; p < SP; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int col = group * SC + p * 16 + 2 * j;
          const float inv = scale_inverse(ss);
          if (col < a.dk) a.state_out[sat + (long long)col * a.dv] = S[p][j].x * inv;
          if (col + 1 < a.dk) a.state_out[sat + (long long)(col + 1) * a.dv] = S[p][j].y * inv;
        }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kScanWarps) tmem_free(tm, 512);
}

template <typename T, int DK, bool STAGED>
__global__ void __launch_bounds__(kScanThreads, 1)
delta_scan_kernel(const DeltaArgs a, const DeltaPlan plan, const char *kq, const char *images,
                  int *status) {
  delta_scan<T, DK, false, STAGED>(a, plan, blockIdx.x, kq, images, nullptr, nullptr, nullptr,
                                   status);
}

}  // namespace fftgb
