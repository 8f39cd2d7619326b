// delta_scan.cuh -- the gated delta rule from chunk to chunk (delta.cuh).
//
// One block walks a sequence's chunks for one head and 128 columns of v, with
// everything transposed: a column of v is a lane of tensor memory and a row
// of the left operands, K and Q in shared memory serve as right operands as
// they come (K-major for S^T K^T, MN-major for U^T K).  Per chunk
//   P = S^T K^T, N = S^T Q^T;  Y = V^T - P gamma;  E = Y T^T (T the inverse);
//   U = E beta;  W = U Gamma / gamma;  S^T <- S^T Gamma + W K;
//   O^T = scale (N gamma + U M^T).
// Two threads own a column of v, each with half of the tokens and half of
// the state's columns: the state itself stays in their registers in fp32,
// and what they hand to the tensor cores (S, Y, U, W) is scaled by the power
// of two of the column's largest value, which they agree on through shared
// memory, and split into two fp16 values.  Only P -> Y -> E -> U -> S is a
// chain; N, U M^T, the output and all loads run beside it.
//
// Roles: 8 warps of arithmetic, one thread that issues the products, one
// that fetches the chunks' images ahead (bulk copies, 3 or 2 stages).
//
// Tensor memory (512 columns):
//   W K (fp32)       0 .. DK - 1
//   S (two fp16)     128, 192        P, then E     256 .. 319
//   Y, then U        320, 352        W             384, 416
//   N, then O        448 .. 511
#pragma once

#include "delta.cuh"

namespace fftgb {

constexpr int kScanThreads = 10 * 32;
constexpr int kScanMath = 256;

__host__ __device__ constexpr int scan_stages(int terms) { return terms == 1 ? 3 : 2; }
// Stage: the tiles of K and Q, then the head's image, 1024-byte aligned.
__host__ __device__ constexpr int scan_stage_bytes(int dk, int terms) {
  return kq_bytes(dk, terms) + ((kImageBytes + 1023) & ~1023);
}
__host__ __device__ constexpr size_t scan_smem(int dk, int terms) {
  return 1024 + (size_t)scan_stages(terms) * scan_stage_bytes(dk, terms);
}

struct ScanBars {
  uint64_t full[3], empty[3];
  uint64_t p, n, e, s, o;       // products done: P, N, E, W K, O
  uint64_t y, u, ns, sb, of;    // operands ready: Y, U and W, N scaled, S; O read
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

// The loading thread: the chunks' images into the stages.
template <int DK, int NT>
__device__ __forceinline__ void scan_load(const DeltaArgs &a, const ScanSpan &sp, int h,
                                          bool backwards, const char *kq, const char *images,
                                          char *stages, ScanBars *bars, volatile int *failed,
                                          int *status) {
  constexpr int ST = scan_stages(NT);
  const int hk = h / (a.vheads / a.kheads);
  int issued = 0;
  for (int it = 0; it < sp.chunks; ++it) {
    const long long c = sp.chunk0 + (backwards ? sp.chunks - 1 - it : it);
    const int s = it % ST;
    if (it >= ST && !wait_or_fail(&bars->empty[s], (it / ST - 1) & 1, failed, status)) break;
    char *stage = stages + s * scan_stage_bytes(DK, NT);
    bar_arrive_tx(&bars->full[s], kq_bytes(DK, NT) + kImageBytes);
    bulk_load(stage, kq + (c * a.kheads + hk) * (long long)kq_bytes(DK, NT), kq_bytes(DK, NT),
              &bars->full[s]);
    bulk_load(stage + kq_bytes(DK, NT), images + (c * a.vheads + h) * (long long)kImageBytes,
              kImageBytes, &bars->full[s]);
    issued = it + 1;
  }
  // Given up: no copy may land after the block has gone.
  if (*failed)
    for (int it = issued > ST ? issued - ST : 0; it < issued; ++it)
      bar_wait(&bars->full[it % ST], (it / ST) & 1);
}

constexpr uint32_t idesc_tokens = mma_desc(128, 64, false, false);

// S^T X^T into `d` (64 columns): left operand the state's two parts, right
// one the chunk's X (K or Q).  LEAD: leading parts only.
template <int DK, int NT, bool LEAD>
__device__ __forceinline__ void mma_state(uint32_t d, uint32_t hi, uint32_t lo, uint32_t x) {
  constexpr uint32_t kPlane = 2 * (DK / 64) * kTile;
#pragma unroll
  for (int term = 0; term < (LEAD ? 1 : NT == 1 ? 2 : 3); ++term) {
    const uint32_t ta = term == 1 ? lo : hi, tb = x + (term == 2 ? kPlane : 0);
#pragma unroll
    for (int k = 0; k < DK / 16; ++k)
      mma_ts(d, ta + 8 * k, tile_desc(tb + (k >> 2) * 2 * kTile + (k & 3) * 32, 16, 1024),
             idesc_tokens, term > 0 || k > 0);
  }
}
// A B^T for 64-token A (two parts) and a 64 x 64 matrix of the image.
template <bool LEAD>
__device__ __forceinline__ void mma_inner(uint32_t d, uint32_t hi, uint32_t lo, uint32_t m,
                                          bool accumulate) {
#pragma unroll
  for (int term = 0; term < (LEAD ? 1 : 3); ++term) {
    const uint32_t ta = term == 1 ? lo : hi, tb = m + (term == 2 ? kTile : 0);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      mma_ts(d, ta + 8 * k, tile_desc(tb + k * 32, 16, 1024), idesc_tokens,
             accumulate || term > 0 || k > 0);
  }
}
// A X for 64-token A and the chunk's X (K or Q) as 64 tokens x DK.
template <int DK, int NT>
__device__ __forceinline__ void mma_update(uint32_t d, uint32_t hi, uint32_t lo, uint32_t x,
                                           bool accumulate) {
  constexpr uint32_t idesc = mma_desc(128, DK, false, true);
  constexpr uint32_t kPlane = 2 * (DK / 64) * kTile;
#pragma unroll
  for (int term = 0; term < (NT == 1 ? 2 : 3); ++term) {
    const uint32_t ta = term == 1 ? lo : hi, tb = x + (term == 2 ? kPlane : 0);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      mma_ts(d, ta + 8 * k, tile_desc(tb + k * 2048, 2 * kTile, 1024), idesc,
             accumulate || term > 0 || k > 0);
  }
}

// 32 values times s to the two parts of a left operand (16 packed columns each).
__device__ __forceinline__ void put_split(uint32_t hi_at, uint32_t lo_at, const float (&f)[32],
                                          float s) {
  uint32_t hi[16], lo[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) split2(f[2 * j], f[2 * j + 1], s, hi[j], lo[j]);
  tmem_st16(hi_at, hi);
  tmem_st16(lo_at, lo);
}
__device__ __forceinline__ float max32(const float (&f)[32]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 32; ++j) m = fmaxf(m, fabsf(f[j]));
  return m;
}

// One arrival per warp, after every lane's accesses to tensor memory.
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) bar_arrive(bar);
}

// The scale that the two threads of a column of v agree on: each brings the
// largest value of its half.  The two warps meet at a barrier of their own,
// the two halves of `box` alternate, so one barrier per agreement is enough.
struct RowAgree {
  float (*box)[2][128];
  int row, half, pair, turn;
  __device__ __forceinline__ float scale(float m) {
    box[turn][half][row] = m;
    asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory");
    m = fmaxf(m, box[turn][half ^ 1][row]);
    turn ^= 1;
    return row_scale(m);
  }
};

constexpr uint32_t kColD = 0, kColSh = 128, kColSl = 192, kColP = 256, kColYh = 320, kColYl = 352,
                   kColWh = 384, kColWl = 416, kColN = 448;

// Barriers and tensor memory of a scan: returns the base column.
__device__ __forceinline__ uint32_t scan_begin(ScanBars &bars, uint32_t *slot, volatile int *failed,
                                               int tid, int warp) {
  if (warp == 8) tmem_alloc(slot, 512);
  if (tid == 0) {
    for (int s = 0; s < 3; ++s) {
      bar_init(&bars.full[s], 1);
      bar_init(&bars.empty[s], 1 + kScanMath / 32);
    }
    for (uint64_t *b : {&bars.p, &bars.n, &bars.e, &bars.s, &bars.o, &bars.done}) bar_init(b, 1);
    for (uint64_t *b : {&bars.y, &bars.u, &bars.ns, &bars.sb, &bars.of})
      bar_init(b, kScanMath / 32);
    *failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return *slot;
}

// SAVE leaves for the gradients, per chunk, head and 128 columns of v, the
// state that entered the chunk (fp32 [DK][128]) and E (fp32 [64][128]).
template <typename T, int DK, bool SAVE>
__global__ void __launch_bounds__(kScanThreads, 1)
delta_scan_kernel(const DeltaArgs a, const DeltaPlan plan, const char *kq, const char *images,
                  float *states, float *rows, int *status) {
  extern __shared__ char smem_raw[];
  __shared__ ScanBars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int failed;
  __shared__ float box[2][2][128];
  constexpr int NT = Terms<T>::value, ST = scan_stages(NT);
  // bf16 outputs: their rounding (2^-9) hides what the leading fp16 parts of
  // S, U and M leave out (2^-12) in the products that only the output sees.
  constexpr bool LEAD = std::is_same<T, __nv_bfloat16>::value;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int blocks_v = (a.dv + 127) / 128;
  const int vb = blockIdx.x % blocks_v;
  const int h = (blockIdx.x / blocks_v) % a.vheads;
  const ScanSpan sp = scan_span(a, plan, blockIdx.x / blocks_v / a.vheads);
  char *stages = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t tm = scan_begin(bars, &tmem_slot, &failed, tid, warp);
  auto wait = [&](uint64_t *b, uint32_t parity) { return wait_or_fail(b, parity, &failed, status); };

  if (warp == 9) {
    if (lane == 0)
      scan_load<DK, NT>(a, sp, h, false, kq, images, stages, &bars, &failed, status);
    __syncwarp();
  } else if (warp == 8) {
    if (lane == 0) {
      for (int it = 0; it < sp.chunks; ++it) {
        const int s = it % ST;
        const uint32_t ph = it & 1;
        const uint32_t k = smem_u32(stages + s * scan_stage_bytes(DK, NT));
        const uint32_t q = k + kTile, image = k + kq_bytes(DK, NT);
        if (!wait(&bars.full[s], (it / ST) & 1) || !wait(&bars.sb, ph)) break;
        tc_fence_after();
        mma_state<DK, NT, false>(tm + kColP, tm + kColSh, tm + kColSl, k);
        mma_commit(&bars.p);
        if (it > 0 && !wait(&bars.of, ph ^ 1)) break;
        tc_fence_after();
        mma_state<DK, NT, LEAD>(tm + kColN, tm + kColSh, tm + kColSl, q);
        mma_commit(&bars.n);
        if (!wait(&bars.y, ph)) break;
        tc_fence_after();
        mma_inner<false>(tm + kColP, tm + kColYh, tm + kColYl, image, false);
        mma_commit(&bars.e);
        if (!wait(&bars.u, ph)) break;
        tc_fence_after();
        mma_update<DK, NT>(tm + kColD, tm + kColWh, tm + kColWl, k, false);
        mma_commit(&bars.s);
        if (!wait(&bars.ns, ph)) break;
        tc_fence_after();
        mma_inner<LEAD>(tm + kColN, tm + kColYh, tm + kColYl, image + 2 * kTile, true);
        mma_commit(&bars.o);
        mma_commit(&bars.empty[s]);
      }
      mma_commit(&bars.done);
      bar_wait(&bars.done, 0);
    }
    __syncwarp();
  } else {
    const int half = warp >> 2;              // tokens and state columns of this group
    const int row = (warp & 3) * 32 + lane;  // column of v within the block
    const uint32_t lb = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const int dvr = vb * 128 + row;
    const bool live = dvr < a.dv;
    constexpr int SC = DK / 2;               // state columns of a thread
    const long long sat = ((sp.b * a.vheads + h) * a.dk) * (long long)a.dv + dvr;
    RowAgree agree{box, row, half, warp & 3, 0};
    auto saved = [&](long long c) { return ((sp.chunk0 + c) * a.vheads + h) * blocks_v + vb; };
    auto gates_of = [&](int s) {
      return reinterpret_cast<const float *>(stages + s * scan_stage_bytes(DK, NT) +
                                             kq_bytes(DK, NT) + 4 * kTile);
    };
    float vr[32];
    auto fetch_v = [&](int c) {
      const long long r0 = sp.row0 + (long long)c * kChunk + half * 32;
      const long long left = sp.rows - (long long)c * kChunk - half * 32;
      const T *v = head_rows<T>(a.v, a.sv, sp.b, r0, h) + dvr;
#pragma unroll
      for (int j = 0; j < 32; ++j) vr[j] = live && j < left ? to_acc(v[j * a.sv.tok]) : 0.0f;
    };
    float S[SC / 32][32], inv_s = 1.0f;
    // The state as the left operand of chunk c's products.
    auto put_state = [&](long long c) {
      float m = max32(S[0]);
      if constexpr (SC > 32) m = fmaxf(m, max32(S[SC / 32 - 1]));
      const float s = agree.scale(m);
      inv_s = scale_inverse(s);
#pragma unroll
      for (int p = 0; p < SC / 32; ++p) {
        const int col = half * SC + p * 32;
        put_split(lb + kColSh + col / 2, lb + kColSl + col / 2, S[p], s);
      }
      tmem_wait_st();
      warp_arrive(&bars.sb, lane);
      if constexpr (SAVE) {
        float *dst = states + saved(c) * (DK * 128) + row;
#pragma unroll
        for (int p = 0; p < SC / 32; ++p)
#pragma unroll
          for (int j = 0; j < 32; ++j) dst[(half * SC + p * 32 + j) * 128] = S[p][j];
      }
    };
#pragma unroll
    for (int p = 0; p < SC / 32; ++p)
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const int col = half * SC + p * 32 + j;
        S[p][j] = a.state_in && live && col < a.dk ? a.state_in[sat + (long long)col * a.dv] : 0.0f;
      }
    bool ok = true;
    if (sp.chunks > 0) {
      fetch_v(0);
      put_state(0);
    }
    for (int it = 0; it < sp.chunks && ok; ++it) {
      const int s = it % ST;
      const uint32_t ph = it & 1;
      const float *gates = gates_of(s) + half * 32;
      uint32_t r[32];
      float f[32];
      // Y = V^T - P gamma
      if (!(ok = wait(&bars.full[s], (it / ST) & 1) && wait(&bars.p, ph))) break;
      tc_fence_after();
      tmem_ld32(lb + kColP + half * 32, r);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; ++j) f[j] = vr[j] - gates[j] * inv_s * __uint_as_float(r[j]);
      const float ys = agree.scale(max32(f));
      put_split(lb + kColYh + half * 16, lb + kColYl + half * 16, f, ys);
      tmem_wait_st();
      warp_arrive(&bars.y, lane);
      // U = E beta, W = U Gamma / gamma
      if (!(ok = wait(&bars.e, ph))) break;
      tc_fence_after();
      tmem_ld32(lb + kColP + half * 32, r);
      tmem_wait_ld();
      const float inv_y = scale_inverse(ys);
#pragma unroll
      for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(r[j]) * (gates[5 * 64 + j] * inv_y);
      if constexpr (SAVE) {
        float *dst = rows + saved(it) * (64 * 128) + half * 32 * 128 + row;
#pragma unroll
        for (int j = 0; j < 32; ++j) dst[j * 128] = f[j];
      }
      float um = 0.0f;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        f[j] *= gates[2 * 64 + j];
        um = fmaxf(um, fmaxf(fabsf(f[j]), fabsf(f[j] * gates[64 + j])));
      }
      const float us = agree.scale(um), inv_u = scale_inverse(us);
      put_split(lb + kColYh + half * 16, lb + kColYl + half * 16, f, us);
#pragma unroll
      for (int j = 0; j < 32; ++j) f[j] *= gates[64 + j];
      put_split(lb + kColWh + half * 16, lb + kColWl + half * 16, f, us);
      tmem_wait_st();
      warp_arrive(&bars.u, lane);
      // N in units of U M^T, the start of O
      if (!(ok = wait(&bars.n, ph))) break;
      tc_fence_after();
      tmem_ld32(lb + kColN + half * 32, r);
      tmem_wait_ld();
      const float ratio = inv_s * us;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        r[j] = __float_as_uint(__uint_as_float(r[j]) * (gates[3 * 64 + j] * ratio));
      tmem_st32(lb + kColN + half * 32, r);
      tmem_wait_st();
      warp_arrive(&bars.ns, lane);
      const float Gamma = gates_of(s)[kGammaAt];
      const bool more = it + 1 < sp.chunks;
      if (more) fetch_v(it + 1);
      // The new state
      if (!(ok = wait(&bars.s, ph))) break;
      tc_fence_after();
#pragma unroll
      for (int p = 0; p < SC / 32; ++p) {
        tmem_ld32(lb + kColD + half * SC + p * 32, r);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) S[p][j] = fmaf(S[p][j], Gamma, __uint_as_float(r[j]) * inv_u);
      }
      if (more) put_state(it + 1);
      // The output
      if (!(ok = wait(&bars.o, ph))) break;
      tc_fence_after();
      tmem_ld32(lb + kColN + half * 32, r);
      tmem_wait_ld();
      warp_arrive(&bars.of, lane);
      if (a.o && live) {
        const long long r0 = sp.row0 + (long long)it * kChunk + half * 32;
        const long long left = sp.rows - (long long)it * kChunk - half * 32;
        T *o = static_cast<T *>(a.o) + out_row(a, sp.b, r0, plan.chunk0 != nullptr, h) + dvr;
        const long long step = (long long)a.vheads * a.dv;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < left)
            o[j * step] = from_acc<T>(__uint_as_float(r[j]) * (gates[4 * 64 + j] * inv_u));
      }
      __syncwarp();
      if (lane == 0) bar_arrive(&bars.empty[s]);  // the gates were read
    }
    if (ok && a.state_out && live) {
#pragma unroll
      for (int p = 0; p < SC / 32; ++p)
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int col = half * SC + p * 32 + j;
          if (col < a.dk) a.state_out[sat + (long long)col * a.dv] = S[p][j];
        }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_free(tm, 512);
}

}  // namespace fftgb
