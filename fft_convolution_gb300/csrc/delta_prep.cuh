// delta_prep.cuh -- what the scans of the gated delta rule need of each
// chunk (delta.cuh): K and Q as scaled fp16 tiles, the inverse of the unit
// triangular matrix, M, and the factors of its tokens.
//
// One block per chunk and key head.  [K; Q] K^T (128 x 64) is one product on
// the tensor cores, kept in tensor memory for all value heads that share the
// key head; each of the 128 threads then owns one row of it.  With A the
// strictly lower triangular matrix of delta.cuh and R = (I + A beta)^-1 A,
//   (I + A beta)^-1 = I - R beta  and  (I + beta A)^-1 = I - beta R,
// so one R serves both scans.  It is taken in fp32: the four 16 x 16 diagonal
// blocks by substitution (one warp each, one column per lane), the blocks
// below them by products, doubling the solved size twice:
//   R_21 = (I - R_22 beta_2) A_21 (I - beta_1 R_11).
// Substitution alone would be a chain of 64 dependent steps, and a power
// series of A would cancel catastrophically for keys that repeat.
//
// Shared memory's latency bounds it: five blocks of four warps per SM (registers
// and shared memory) issue 39% of the time (49% without the second image).  8192
// tokens with 16 key and 32 value heads of 128 x 128 take 110 us, 16384 tokens of
// 16 heads with the images for both directions, which spill 124 bytes per thread
// in bf16, 205 (2.6 TB/s).
//
// Everything is written in exactly the layout of the scans' shared memory,
// so they fetch a chunk with two bulk copies, whatever the inputs' type,
// strides and alignment.
//
// Forward image: (I + A beta)^-1 and M by rows; per token
//   0: -gamma 2^ek   1: Gamma/gamma beta 2^(ek + et)   2: beta 2^et   3: scale gamma 2^eq
//   4: scale 2^em    5: 2^et
// BACK image: (I + beta A)^-T and M^T; per token
//   0: Gamma/gamma 2^ek   1: scale 2^em   2: 2^et   3: beta
//   4: -gamma beta 2^(ek + et)   5: scale gamma 2^eq
// and in both 6: 2^ek, 7: 2^eq,
// where 2^-e is the scale of a token's row of K (ek), Q (eq), of the inverse
// (et) and of M (em).
//
// Of the chunk: 0: Gamma, then bounds from which the scans choose the scales
// of what they compute without looking at it first.  With |S| the largest
// value of the state in a column of v, K's scaled rows below 2, c = 2 DK, and of
// the inverse's rows r the sums of absolute values and t the same sums weighted
// with gamma 2^ek (BACK: Gamma/gamma 2^ek) of their columns:
//   forward  |Y| <= |V| + b1 |S|,         b1 = max c gamma 2^ek
//            |U| <= b2 |V| + b5 |S|,      b2 = max beta r,  b5 = max c beta t
//            |W| <= b3 |V| + b6 |S|,      the same times Gamma/gamma 2^ek
//            |E| <= b4 |V| + b7 |S|,      b4 = max r,  b7 = max c t
//   BACK     |dU| <= b1 |dS| + b2 |dO|,   b1 = max c Gamma/gamma 2^ek,
//                                         b2 = max scale (row sums of |M^T|)
//            |F| <= b3 b2 |dO| + b6 |dS|, b3 = max r,  b6 = max c t
//            |gamma beta F 2^ek| <= b4 b2 |dO| + b7 |dS|,  the same times gamma beta 2^ek
//            |scale gamma dO 2^eq| <= b5 |dO|
// t, not r times the largest weight: what a decay drops within the chunk must not
// set the scale of what comes behind it.
#pragma once

#include "delta.cuh"

namespace fftgb {

constexpr int kPrepThreads = 128;
constexpr int kPitch = 68;  // floats per row of a 64 x 64 fp32 matrix (rows stay 16-byte aligned)

// The tiles, and in their place (after the product) the two fp32 matrices.
template <typename T, int DK> constexpr size_t prep_smem() {
  constexpr int tiles = kq_bytes(DK, Terms<T>::value), fp32 = 2 * 64 * kPitch * 4;
  return 1024 + (size_t)(tiles > fp32 ? tiles : fp32);
}

// A 64 x 64 lower triangular fp32 matrix m (what lies above its diagonal is
// not read), or its transpose (TRANS), to the leading and trailing tile, rows
// scaled; the rows' inverse scales go to `inv`, the sums of their absolute
// values to `sum`.  INV: of m = R the inverse, I - R beta, or (TRANS) the
// transpose of I - beta R; the sums weighted with `reach` to `far`.
template <bool TRANS, bool INV>
__device__ __forceinline__ void write_image(const float *m, const float *beta, const float *reach,
                                            char *dst, float *inv, float *sum, float *far,
                                            int tid) {
#pragma unroll
  for (int i = tid; i < 64 * 8; i += kPrepThreads) {
    const int r = i >> 3, c = i & 7;
    float f[8];
    if constexpr (TRANS) {
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = m[(c * 8 + k) * kPitch + r];
    } else {
      const float4 x = *reinterpret_cast<const float4 *>(m + r * kPitch + c * 8);
      const float4 y = *reinterpret_cast<const float4 *>(m + r * kPitch + c * 8 + 4);
      f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
      f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
    }
    if constexpr (INV) {
      const float4 x = *reinterpret_cast<const float4 *>(beta + c * 8);
      const float4 y = *reinterpret_cast<const float4 *>(beta + c * 8 + 4);
      f[0] *= -x.x; f[1] *= -x.y; f[2] *= -x.z; f[3] *= -x.w;
      f[4] *= -y.x; f[5] *= -y.y; f[6] *= -y.z; f[7] *= -y.w;
    }
    const int d = r - c * 8;  // the diagonal's place among the eight
    float t = 0.0f, w = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (TRANS ? k < d : k > d) f[k] = 0.0f;
      if (INV && k == d) f[k] = 1.0f;
      t += fabsf(f[k]);
    }
    if constexpr (INV) {
      const float4 x = *reinterpret_cast<const float4 *>(reach + c * 8);
      const float4 y = *reinterpret_cast<const float4 *>(reach + c * 8 + 4);
      w = fmaf(fabsf(f[0]), x.x, fmaf(fabsf(f[1]), x.y, fmaf(fabsf(f[2]), x.z, fabsf(f[3]) * x.w)));
      w = fmaf(fabsf(f[4]), y.x, fmaf(fabsf(f[5]), y.y, fmaf(fabsf(f[6]), y.z, fmaf(fabsf(f[7]), y.w, w))));
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      t += __shfl_xor_sync(0xffffffffu, t, o);
      if constexpr (INV) w += __shfl_xor_sync(0xffffffffu, w, o);
    }
    const float s = row_scale(lane_max<8>(max8(f)));
    if (c == 0) {
      inv[r] = scale_inverse(s);
      sum[r] = t;
      if constexpr (INV) far[r] = w;
    }
    uint4 hi, lo;
    split8(f, s, hi, lo);
    const int at = piece_at(r, c, 0);
    *reinterpret_cast<uint4 *>(dst + at) = hi;
    *reinterpret_cast<uint4 *>(dst + kTile + at) = lo;
  }
}

// G_i of the 64 tokens times log2(e), as the sum of two floats: differences of
// running sums of up to 64 * 128 keep fp32 accuracy.
__device__ __forceinline__ void running_decay(const float *g, long long step, int n, int tid,
                                              double *carry, float2 *out) {
  float x = 0.0f;
  if (tid < 64 && tid < n) {
    x = g[tid * step];
    x = x < kMinLogDecay ? kMinLogDecay : x;  // a NaN stays
  }
  double s = x;
  const int lane = tid & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  if (tid == 31) *carry = s;
  __syncthreads();
  if (tid < 64) {
    if (tid >= 32) s += *carry;
    s *= 1.4426950408889634;
    const float h = (float)s;
    out[tid] = make_float2(h, (float)(s - (double)h));
  }
}
// The same by one warp, two tokens per lane.
__device__ __forceinline__ void running_decay_warp(const float *g, long long step, int n, int lane,
                                                   float2 *out) {
  double x[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int t = 2 * lane + k;
    float v = t < n ? g[t * step] : 0.0f;
    v = v < kMinLogDecay ? kMinLogDecay : v;
    x[k] = v;
  }
  double s = x[0] + x[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const double e = (k ? s : s - x[1]) * 1.4426950408889634;
    const float h = (float)e;
    out[2 * lane + k] = make_float2(h, (float)(e - (double)h));
  }
}
__device__ __forceinline__ float decay_between(float2 i, float2 j) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"((i.x - j.x) + (i.y - j.y)));
  return e;
}

// Rows 0 .. 63 of K or Q into its tiles in shared memory and in the image;
// inv: the rows' inverse scales.  All loads of a thread are issued before any
// value is looked at (half of them with fp32).
template <typename T, int DK>
__device__ __forceinline__ void load_rows(const T *src, long long stride, int n, int cols, bool vec,
                                          char *tiles, char *image, float *inv, int tid) {
  constexpr int P = DK / 8, PER = 64 * P / kPrepThreads, B = sizeof(T) == 2 ? PER : PER / 2;
  constexpr int kPlane = 2 * (DK / 64) * kTile;
#pragma unroll 1
  for (int k0 = 0; k0 < PER; k0 += B) {
    Row8<T> x[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int i = (k0 + k) * kPrepThreads + tid, r = i / P, c = i % P;
      x[k].load(src + (r < n ? r : 0) * stride + c * 8, r < n ? cols - c * 8 : 0, vec);
    }
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int i = (k0 + k) * kPrepThreads + tid, r = i / P, c = i % P;
      float f[8];
      x[k].get(f);
      const float s = row_scale(lane_max<P>(max8(f)));
      if (c == 0) inv[r] = scale_inverse(s);
      uint4 hi, lo;
      split8(f, s, hi, lo);
      const int at = piece_at(r, c, 2 * kTile);
      *reinterpret_cast<uint4 *>(tiles + at) = hi;
      *reinterpret_cast<uint4 *>(image + at) = hi;
      if constexpr (Terms<T>::value == 2) {
        *reinterpret_cast<uint4 *>(tiles + kPlane + at) = lo;
        *reinterpret_cast<uint4 *>(image + kPlane + at) = lo;
      }
    }
  }
}

// z -= P (beta X): ROWS rows of one column, SIZE summed indexes; p points at
// the first of the rows, x at the column, beta at the first summed index.
template <int SIZE, int ROWS>
__device__ __forceinline__ void block_product(const float *p, const float *x, const float *beta,
                                              float (&z)[ROWS]) {
#pragma unroll 2
  for (int k = 0; k < SIZE; k += 4) {
    const float4 b = *reinterpret_cast<const float4 *>(beta + k);
    const float x0 = b.x * x[k * kPitch], x1 = b.y * x[(k + 1) * kPitch];
    const float x2 = b.z * x[(k + 2) * kPitch], x3 = b.w * x[(k + 3) * kPitch];
#pragma unroll
    for (int o = 0; o < ROWS; ++o) {
      const float4 l = *reinterpret_cast<const float4 *>(p + o * kPitch + k);
      z[o] = fmaf(-l.x, x0, fmaf(-l.y, x1, fmaf(-l.z, x2, fmaf(-l.w, x3, z[o]))));
    }
  }
}
// R_21 for the pairs of SIZE x SIZE diagonal blocks: Z = A_21 (I - beta_1 R_11),
// R_21 = Z - R_22 beta_2 Z.
template <int SIZE>
__device__ __forceinline__ void join_blocks(const float *A, float *R, const float *beta, int tid) {
  constexpr int PAIRS = 32 / SIZE, PER = kPrepThreads / PAIRS, ROWS = SIZE * SIZE / PER;
  const int pr = tid / PER, t = tid % PER;
  const int lo = pr * 2 * SIZE, hi = lo + SIZE;
  const int col = t % SIZE, rb = (t / SIZE) * ROWS;
  float z[ROWS];
  const float *a21 = A + (hi + rb) * kPitch + lo;
#pragma unroll
  for (int o = 0; o < ROWS; ++o) z[o] = a21[o * kPitch + col];
  block_product<SIZE, ROWS>(a21, R + lo * kPitch + lo + col, beta + lo, z);
  float *out = R + (hi + rb) * kPitch + lo + col;
#pragma unroll
  for (int o = 0; o < ROWS; ++o) out[o * kPitch] = z[o];
  __syncthreads();
  block_product<SIZE, ROWS>(R + (hi + rb) * kPitch + hi, R + hi * kPitch + lo + col, beta + hi, z);
  __syncthreads();
#pragma unroll
  for (int o = 0; o < ROWS; ++o) out[o * kPitch] = z[o];
  __syncthreads();
}

// GRAD: the images of both scans.
template <typename T, int DK, bool GRAD>
__global__ void __launch_bounds__(kPrepThreads, 5)
delta_prep_kernel(const DeltaArgs a, const DeltaPlan plan, char *kq, char *images, char *back,
                  int *status) {
  extern __shared__ char smem_raw[];
  __shared__ uint64_t bar;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int failed;
  __shared__ double carry;
  __shared__ float2 G[64];
  __shared__ float4 Gk[64];  // G, the scale of K's row
  __shared__ __align__(16) float beta_s[64];
  __shared__ float inv_kq[2 * 64], inv[4][64], sum[4][64], far[2][64];
  __shared__ __align__(16) float reach[2][64];  // gamma 2^ek, Gamma/gamma 2^ek
  __shared__ float most[2][14];
  constexpr int NT = Terms<T>::value;
  constexpr uint32_t kPlane = 2 * (DK / 64) * kTile;  // [K; Q], one term

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.x % a.kheads;
  const long long ci = blockIdx.x / a.kheads;
  DeltaChunk c;
  if (!delta_chunk(a, plan, ci, c)) return;
  // First of all: the next block of this kernel starts on the multiprocessor
  // only when this one has given back the right to allocate.
  if (warp == 0) tmem_alloc(&tmem_slot, 64);

  // Tiles: 128 rows (K above Q) of 64 columns, kTile * 2 bytes each.
  char *tiles = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  float *L = reinterpret_cast<float *>(tiles);
  float *X = L + 64 * kPitch;
  const uint32_t t0 = smem_u32(tiles);
  char *kqi = kq + (ci * a.kheads + hk) * (long long)kq_bytes(DK, NT);
  load_rows<T, DK>(head_rows<T>(a.k, a.sk, c.b, c.row, hk), a.sk.tok, c.n, a.dk,
                   vec_rows<T>(a.k, a.sk), tiles, kqi, inv_kq, tid);
  load_rows<T, DK>(head_rows<T>(a.q, a.sq, c.b, c.row, hk), a.sq.tok, c.n, a.dk,
                   vec_rows<T>(a.q, a.sq), tiles + kTile, kqi + kTile, inv_kq + 64, tid);
  if (tid == 0) {
    bar_init(&bar, 1);
    failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  fence_smem_to_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t acc = __shfl_sync(0xffffffffu, tmem_slot, 0);
  if (warp == 0 && elect_one()) {
    constexpr uint32_t idesc = mma_desc(128, 64, false, false);
#pragma unroll
    for (int term = NT == 1 ? 0 : 2; term >= 0; --term) {
      // trailing x leading, leading x trailing, leading x leading
      const uint32_t ta = t0 + (term == 2 ? kPlane : 0), tb = t0 + (term == 1 ? kPlane : 0);
#pragma unroll
      for (int k = 0; k < DK / 16; ++k) {
        const uint32_t at = (k >> 2) * 2 * kTile + (k & 3) * 32;
        mma_ss(acc, tile_desc(ta + at, 16), tile_desc(tb + at, 16), idesc,
               term < (NT == 1 ? 0 : 2) || k > 0);
      }
    }
    mma_commit(&bar);
  }
  __syncwarp();
  const bool ok = wait_or_fail(&bar, 0, &failed, status);
  if (__syncthreads_and(ok)) {
    tc_fence_after();
    const int group = a.vheads / a.kheads;
    for (int hv = hk * group; hv < (hk + 1) * group; ++hv) {
      char *image = images + (ci * a.vheads + hv) * (long long)kImageBytes;
      const float *g = a.g + c.b * a.sg.seq + c.row * a.sg.tok + hv * a.sg.head;
      const float *beta = a.beta + c.b * a.sb.seq + c.row * a.sb.tok + hv * a.sb.head;
      running_decay(g, a.sg.tok, c.n, tid, &carry, G);
      if (tid < 64) {
        beta_s[tid] = tid < c.n ? beta[tid * a.sb.tok] : 0.0f;
        Gk[tid] = make_float4(G[tid].x, G[tid].y, inv_kq[tid], 0.0f);
      }
      __syncthreads();
      // Row i of A (threads 0 .. 63, from K K^T) or of M (64 .. 127), up to
      // its diagonal (what lies above is arbitrary).
      const int i = tid & 63;
      const float2 gi = G[i];
      const float fi = inv_kq[tid];
      if (tid < 64) {
        reach[0][i] = decay_between(gi, make_float2(0.0f, 0.0f)) * fi;
        if constexpr (GRAD) reach[1][i] = decay_between(G[63], gi) * fi;
      }
      float *row = (tid >= 64 ? X : L) + i * kPitch;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (half == 1 && (warp & 1) == 0) break;  // rows 0 .. 31 end before column 32
        uint32_t r[32];
        tmem_ld(acc + ((uint32_t)(warp * 32) << 16) + half * 32, r);
        tmem_wait_ld();
#pragma unroll
        for (int jj = 0; jj < 32; jj += 4) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 gj = Gk[half * 32 + jj + e];
            x[e] = decay_between(gi, make_float2(gj.x, gj.y)) *
                   (__uint_as_float(r[jj + e]) * (fi * gj.z));
          }
          *reinterpret_cast<float4 *>(row + half * 32 + jj) = make_float4(x[0], x[1], x[2], x[3]);
        }
      }
      __syncthreads();
      char *imageb = back + (ci * a.vheads + hv) * (long long)kImageBytes;
      write_image<false, false>(X, beta_s, nullptr, image + 2 * kTile, inv[1], sum[1], nullptr, tid);
      if constexpr (GRAD)
        write_image<true, false>(X, beta_s, nullptr, imageb + 2 * kTile, inv[3], sum[3], nullptr, tid);
      __syncthreads();
      // Diagonal blocks of R: column `col` of block `warp`, R_m = A_m - sum_p
      // A_mp beta_p R_p; both halves of the warp do the same columns.
      {
        const int col = lane & 15, r0 = warp * 16;
        const float *l = L + r0 * kPitch + r0;
        float x[16];  // beta R
#pragma unroll
        for (int m = 0; m < 16; ++m) {
          float s = m > col ? l[m * kPitch + col] : 0.0f;
#pragma unroll
          for (int p = 0; p < m; p += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(l + m * kPitch + p);
            s = fmaf(-v.x, x[p], s);
            if (p + 1 < m) s = fmaf(-v.y, x[p + 1], s);
            if (p + 2 < m) s = fmaf(-v.z, x[p + 2], s);
            if (p + 3 < m) s = fmaf(-v.w, x[p + 3], s);
          }
          x[m] = s * beta_s[r0 + m];
          // the other half of the warp: zeros right of the first of two blocks
          if (lane < 16) X[(r0 + m) * kPitch + r0 + col] = s;
          else if ((warp & 1) == 0) X[(r0 + m) * kPitch + r0 + 16 + col] = 0.0f;
        }
      }
      __syncthreads();
      join_blocks<16>(L, X, beta_s, tid);
      join_blocks<32>(L, X, beta_s, tid);
      write_image<false, true>(X, beta_s, reach[0], image, inv[0], sum[0], far[0], tid);
      if constexpr (GRAD)
        write_image<true, true>(X, beta_s, reach[1], imageb, inv[2], sum[2], far[1], tid);
      __syncthreads();
      if (tid < 64) {
        float *gates = reinterpret_cast<float *>(image + 4 * kTile) + tid;
        const float ek = inv_kq[tid], eq = inv_kq[64 + tid], em = inv[1][tid], et = inv[0][tid];
        const float gam = decay_between(G[tid], make_float2(0.0f, 0.0f));
        const float dec = decay_between(G[63], G[tid]), bt = beta_s[tid];
        const float ga[kGates] = {-gam * ek, dec * bt * ek * et, bt * et, a.scale * gam * eq,
                                  a.scale * em, et, ek, eq};
        const float ab = fabsf(bt), sc = fabsf(a.scale), t = 2.0f * DK * far[0][tid];
        float b[14];
        b[0] = 2.0f * DK * gam * ek;
        b[1] = ab * sum[0][tid];
        b[2] = b[1] * (dec * ek);
        b[3] = sum[0][tid];
        b[4] = ab * t;
        b[5] = b[4] * (dec * ek);
        b[6] = t;
#pragma unroll
        for (int k = 0; k < kGates; ++k) gates[k * 64] = ga[k];
        if (tid == 63) gates[kChunkAt - 63] = gam;
        if constexpr (GRAD) {
          gates = reinterpret_cast<float *>(imageb + 4 * kTile) + tid;
          const float gb[kGates] = {dec * ek, a.scale * inv[3][tid], inv[2][tid], bt,
                                    -gam * bt * ek * inv[2][tid], a.scale * gam * eq, ek, eq};
#pragma unroll
          for (int k = 0; k < kGates; ++k) gates[k * 64] = gb[k];
          if (tid == 63) gates[kChunkAt - 63] = gam;
          const float gbk = gam * ab * ek, tb = 2.0f * DK * far[1][tid];
          b[7] = 2.0f * DK * dec * ek;
          b[8] = sc * sum[3][tid];
          b[9] = sum[2][tid];
          b[10] = gbk * sum[2][tid];
          b[11] = sc * gam * eq;
          b[12] = tb;
          b[13] = gbk * tb;
        }
        // (of values that are not negative the bits are in order)
#pragma unroll
        for (int k = 0; k < (GRAD ? 14 : 7); ++k) {
          const unsigned m = __reduce_max_sync(0xffffffffu, __float_as_uint(b[k]));
          if (lane == 0) most[warp][k] = __uint_as_float(m);
        }
      }
      __syncthreads();
      if (tid < (GRAD ? 14 : 7))
        reinterpret_cast<float *>((tid < 7 ? image : imageb) + 4 * kTile)
            [kChunkAt + 1 + (tid < 7 ? tid : tid - 7)] = fmaxf(most[0][tid], most[1][tid]);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 0) tmem_free(acc, 64);
}

}  // namespace fftgb
