// delta_grad.cuh -- dq, dk, dg and dbeta of the gated delta rule, all chunks in
// parallel, from what the two scans left (delta.cuh): the state S0 that
// entered the chunk, the gradient dS of the state that left it, E and F.
//
// With X_ij = [j <= i] scale D_ij beta_j dO_i . E_j and
//      Z_ij = -[j < i] D_ij beta_i beta_j F_i . E_j:
//   dQ  = scale gamma (dO S0^T) + X K
//   dKr = Z K - gamma beta (F S0^T)                  (K as what is read under)
//   dKw = Gamma/gamma beta (E dS^T) + X^T Q + Z^T K  (K as what is written under)
//   dbeta_i = E_i . F_i
//   dG_i = q_i . dQ_i + k_i . (dKr_i - dKw_i), and <S1, dS> at the chunk's end,
//   dg_i = dG_i + dG_{i+1} + ... to the chunk's end
// (every place where a token's q or k enters carries its e^{G_i}, every one
// where k is written under its e^{-G_i}); <S1, dS> = Gamma <S0, dS> +
// sum_j k_j . (Gamma/gamma beta dS E)_j.
//
// One block per chunk and value head, products transposed (dk along the lanes
// of tensor memory, tokens along the columns): S0 and dS are left operands,
// dO, F and E right ones, [dO; F] E^T one product of 128 rows; then K and Q
// (MN-major) on the left, X and Z on the right.  Heads that share a key head
// leave fp32 partial sums, added by a small kernel in a fixed order.
//
// Reading S0, dS, E and F (192 KB for 128 x 128 heads) bounds it.
#pragma once

#include "delta_prep.cuh"
#include "delta_scan.cuh"

namespace fftgb {

constexpr int kGradThreads = 512;
// S0 / dS (two parts), later X and Z; [dO; F] (two parts), later K and Q; E.
constexpr int kGradA = 4 * 128 * 128, kGradB = 8 * kTile, kGradC = 4 * kTile;
constexpr size_t grad_smem() { return 1024 + kGradA + kGradB + kGradC; }

struct GradShared {
  uint64_t mma, kq;
  uint32_t tmem_slot;
  int failed;
  float2 G[64];
  double carry;
  float beta[64], gam[64], dec[64], ek[64], eq[64];
  // inverse scales of the rows of S0, dS, [dO; F] and E
  float s0[128], ds[128], of[128], e[64];
  unsigned most[4];       // largest X1, Z1, and X2 or Z2
  float dots[4][64];
  float part[2][16];
};

// Rows of 128 columns, four per lane: the largest value of a row, over all
// blocks of columns when there are several.
__device__ __forceinline__ float4 load4(const float *p, int col, int dv, bool there) {
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (there) x = *reinterpret_cast<const float4 *>(p);
  if (col + 3 >= dv) {
    if (col >= dv) x.x = 0.0f;
    if (col + 1 >= dv) x.y = 0.0f;
    if (col + 2 >= dv) x.z = 0.0f;
    x.w = 0.0f;
  }
  return x;
}
template <typename T>
__device__ __forceinline__ float4 load4(const T *p, int left, bool vec, bool there) {
  float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (there) {
    if (vec && left >= 4) {
      T t[4];
      if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4 *>(t) = *reinterpret_cast<const uint4 *>(p);
      else *reinterpret_cast<uint2 *>(t) = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = to_acc(t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) f[i] = to_acc(p[i]);
    }
  }
  return make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ float max4(float4 x) {
  return fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
}
// A lane's four values of row r to the two parts of the tiles.
__device__ __forceinline__ void put4(char *hi_tiles, int lo_at, int tile, int r, int lane, float4 x,
                                     float s) {
  uint2 hi, lo;
  split2(mul2(make_float2(x.x, x.y), both(s)), hi.x, lo.x);
  split2(mul2(make_float2(x.z, x.w), both(s)), hi.y, lo.y);
  const int at = piece_at(r, lane >> 1, tile) + (lane & 1) * 8;
  *reinterpret_cast<uint2 *>(hi_tiles + at) = hi;
  *reinterpret_cast<uint2 *>(hi_tiles + lo_at + at) = lo;
}

// A (shared, 128 rows, `ablock` bytes between tiles of 64 columns, trailing
// parts `alo` bytes on) times B (64 rows) over 128 columns.
__device__ __forceinline__ void mma_cols(uint32_t d, uint32_t a, uint32_t ablock, uint32_t alo,
                                         uint32_t b, uint32_t bblock, uint32_t blo, bool b_exact,
                                         bool accumulate) {
  constexpr uint32_t idesc = mma_desc(128, 64, false, false);
#pragma unroll
  for (int term = 2; term >= 0; --term) {  // trailing parts first (delta_scan.cuh)
    if (term == 2 && b_exact) continue;
    const uint32_t ta = a + (term == 1 ? alo : 0), tb = b + (term == 2 ? blo : 0);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      mma_ss(d, tile_desc(ta + (k >> 2) * ablock + (k & 3) * 32, 16),
             tile_desc(tb + (k >> 2) * bblock + (k & 3) * 32, 16), idesc,
             accumulate || term < (b_exact ? 1 : 2) || k > 0);
  }
}
// K^T or Q^T (MN-major, 64 tokens) times a 64 x 64 matrix in two parts,
// K-major (rows = columns of the result) or MN-major (B_MN).
template <int DK, int NT, bool B_MN>
__device__ __forceinline__ void mma_tokens(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
  constexpr uint32_t idesc = mma_desc(128, 64, true, B_MN);
  constexpr uint32_t kPlane = 2 * (DK / 64) * kTile;
  constexpr uint32_t block = DK == 128 ? 2 * kTile : 0;  // DK = 64: lanes 64 .. 127 repeat
#pragma unroll
  for (int term = NT == 1 ? 1 : 2; term >= 0; --term) {
    const uint32_t ta = a + (term == 2 ? kPlane : 0), tb = b + (term == 1 ? kTile : 0);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      mma_ss(d, tile_desc(ta + k * 2048, block), tile_desc(tb + (B_MN ? k * 2048 : k * 32), 16),
             idesc, accumulate || term < (NT == 1 ? 1 : 2) || k > 0);
  }
}

constexpr uint32_t kColQ1 = 0, kColR1 = 64, kColW1 = 128, kColG = 192, kColQ2 = 256, kColR2 = 320,
                   kColW2 = 384;

// Sums of 16 values per lane over the warp: lane l gets that of value l >> 1.
__device__ __forceinline__ float warp_sums(float (&v)[16], int lane) {
#pragma unroll
  for (int w = 8, o = 16; w >= 1; w >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float give = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// PARTIAL: dq and dk of this value head go to `partial` (fp32 [2][64][DK] in
// place of the block's E and F), else to their arrays.
template <typename T, int DK, bool PARTIAL>
__global__ void __launch_bounds__(kGradThreads, 1)
delta_grad_kernel(const DeltaArgs a, const DeltaGradArgs ga, const DeltaPlan plan, const char *kq,
                  const char *back, const float *states, const float *dstates, float *es,
                  float *fs, int *status) {
  extern __shared__ char smem_raw[];
  __shared__ GradShared sh;
  constexpr int NT = Terms<T>::value;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int h = blockIdx.x % a.vheads, hk = h / (a.vheads / a.kheads);
  const long long ci = blockIdx.x / a.vheads;
  DeltaChunk c;
  if (!delta_chunk(a, plan, ci, c)) return;
  char *ra = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  char *rb = ra + kGradA, *rc = rb + kGradB;
  const int blocks_v = (a.dv + 127) / 128;
  const long long slot = (ci * a.vheads + h) * blocks_v;
  const bool packed = plan.chunk0 != nullptr;
  volatile int *failed = &sh.failed;

  if (warp == 0) tmem_alloc(&sh.tmem_slot, 512);
  if (tid == 0) {
    bar_init(&sh.mma, 1);
    bar_init(&sh.kq, 1);
    sh.failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < 4) sh.most[tid] = 0;
  if (tid < 128) sh.s0[tid] = sh.ds[tid] = sh.of[tid] = 0.0f;
  if (tid < 64) sh.e[tid] = 0.0f;
  {
    const float *gates = reinterpret_cast<const float *>(
        back + (ci * a.vheads + h) * (long long)kImageBytes + 4 * kTile);
    if (tid < 64) {
      sh.beta[tid] = gates[3 * 64 + tid];
      sh.ek[tid] = gates[6 * 64 + tid];
      sh.eq[tid] = gates[7 * 64 + tid];
    }
  }
  running_decay(a.g + c.b * a.sg.seq + c.row * a.sg.tok + h * a.sg.head, a.sg.tok, c.n, tid,
                &sh.carry, sh.G);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, sh.tmem_slot, 0);
  if (tid < 64) {
    sh.gam[tid] = decay_between(sh.G[tid], make_float2(0.0f, 0.0f));
    sh.dec[tid] = decay_between(sh.G[63], sh.G[tid]);
  }
  const long long orow = out_row(a, c.b, c.row, packed, h), ostep = (long long)a.vheads * a.dv;
  const bool ovec = a.dv % 4 == 0 && ((uintptr_t)ga.dout & 15u) == 0;
  const int col = lane * 4;
  // A warp takes whole rows: its lanes' four values of the row.
  auto row_s = [&](const float *p, int vb, int r) {
    return load4(p + (slot + vb) * (DK * 128) + r * 128 + col, vb * 128 + col, a.dv, true);
  };
  auto row_e = [&](const float *p, int vb, int r) {
    return load4(p + (slot + vb) * (64 * 128) + r * 128 + col, vb * 128 + col, a.dv, r < c.n);
  };
  auto row_o = [&](int vb, int r) {
    const int left = a.dv - vb * 128 - col;
    return load4<T>(static_cast<const T *>(ga.dout) + orow + r * ostep + vb * 128 + col, left, ovec,
                    r < c.n && left > 0);
  };
  // Several blocks of columns: the rows' largest values over all of them first.
  if (blocks_v > 1) {
    for (int vb = 0; vb < blocks_v; ++vb) {
      for (int r = warp; r < DK; r += 16) {
        const float m = lane_max<32>(max4(row_s(states, vb, r)));
        const float n = lane_max<32>(max4(row_s(dstates, vb, r)));
        if (lane == 0) {
          sh.s0[r] = fmaxf(sh.s0[r], m);
          sh.ds[r] = fmaxf(sh.ds[r], n);
        }
      }
      for (int r = warp; r < 64; r += 16) {
        const float m = lane_max<32>(max4(row_o(vb, r))), n = lane_max<32>(max4(row_e(fs, vb, r)));
        const float e = lane_max<32>(max4(row_e(es, vb, r)));
        if (lane == 0) {
          sh.of[r] = fmaxf(sh.of[r], m);
          sh.of[64 + r] = fmaxf(sh.of[64 + r], n);
          sh.e[r] = fmaxf(sh.e[r], e);
        }
      }
    }
    __syncthreads();
    if (tid < 128) {
      sh.s0[tid] = scale_inverse(row_scale(sh.s0[tid]));
      sh.ds[tid] = scale_inverse(row_scale(sh.ds[tid]));
      sh.of[tid] = scale_inverse(row_scale(sh.of[tid]));
    }
    if (tid < 64) sh.e[tid] = scale_inverse(row_scale(sh.e[tid]));
    __syncthreads();
  }
  auto scale_of = [&](float4 x, float *inv) {
    if (blocks_v > 1) return scale_inverse(*inv);
    const float s = row_scale(lane_max<32>(max4(x)));
    __syncwarp();
    if (lane == 0) *inv = scale_inverse(s);
    return s;
  };
  const uint32_t sa = smem_u32(ra), sb = smem_u32(rb), sc = smem_u32(rc);
  uint32_t ph = 0;
  bool ok = true;
  float inner = 0.0f;  // <S0, dS>
  for (int vb = 0; vb < blocks_v && ok; ++vb) {
    constexpr int RS = DK / 16, RT = 4;  // rows of a warp
    {
      float4 x[RS];
#pragma unroll
      for (int k = 0; k < RS; ++k) x[k] = row_s(states, vb, warp + 16 * k);
#pragma unroll
      for (int k = 0; k < RS; ++k) {
        const int r = warp + 16 * k;
        put4(ra, 2 * 128 * 128, 128 * 128, r, lane, x[k], scale_of(x[k], &sh.s0[r]));
      }
    }
    {
      float4 x[RT], y[RT], z[RT];
#pragma unroll
      for (int k = 0; k < RT; ++k) {
        const int r = warp + 16 * k;
        x[k] = row_o(vb, r);
        y[k] = row_e(fs, vb, r);
        z[k] = row_e(es, vb, r);
      }
#pragma unroll
      for (int k = 0; k < RT; ++k) {
        const int r = warp + 16 * k;
        put4(rb, 4 * kTile, 2 * kTile, r, lane, x[k], scale_of(x[k], &sh.of[r]));
        put4(rb, 4 * kTile, 2 * kTile, 64 + r, lane, y[k], scale_of(y[k], &sh.of[64 + r]));
        put4(rc, 2 * kTile, kTile, r, lane, z[k], scale_of(z[k], &sh.e[r]));
      }
    }
    fence_smem_to_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0 && elect_one()) {
      constexpr uint32_t lo_a = 2 * 128 * 128, lo_b = 4 * kTile;
      mma_cols(tm + kColQ1, sa, 128 * 128, lo_a, sb, 2 * kTile, lo_b, NT == 1, vb > 0);
      mma_cols(tm + kColR1, sa, 128 * 128, lo_a, sb + kTile, 2 * kTile, lo_b, false, vb > 0);
      mma_cols(tm + kColG, sb, 2 * kTile, lo_b, sc, kTile, 2 * kTile, false, vb > 0);
      mma_commit(&sh.mma);
    }
    __syncwarp();
    {
      float4 x[RS];
#pragma unroll
      for (int k = 0; k < RS; ++k) x[k] = row_s(dstates, vb, warp + 16 * k);
      ok = wait_or_fail(&sh.mma, ph, failed, status);
      ph ^= 1;
#pragma unroll
      for (int k = 0; k < RS; ++k) {
        // <S0, dS>: S0 from its two parts, before they are overwritten
        const int r = warp + 16 * k;
        const int at = piece_at(r, lane >> 1, 128 * 128) + (lane & 1) * 8;
        const uint2 hi = *reinterpret_cast<const uint2 *>(ra + at);
        const uint2 lo = *reinterpret_cast<const uint2 *>(ra + 2 * 128 * 128 + at);
        auto two = [](uint32_t x) { return __half22float2(*reinterpret_cast<const __half2 *>(&x)); };
        const float2 h0 = two(hi.x), h1 = two(hi.y), l0 = two(lo.x), l1 = two(lo.y);
        inner += sh.s0[r] * ((h0.x + l0.x) * x[k].x + (h0.y + l0.y) * x[k].y +
                             (h1.x + l1.x) * x[k].z + (h1.y + l1.y) * x[k].w);
        put4(ra, 2 * 128 * 128, 128 * 128, r, lane, x[k], scale_of(x[k], &sh.ds[r]));
      }
    }
    fence_smem_to_async();
    tc_fence_before();
    ok = __syncthreads_and(ok);
    tc_fence_after();
    if (ok && warp == 0 && elect_one()) {
      mma_cols(tm + kColW1, sa, 128 * 128, 2 * 128 * 128, sc, kTile, 2 * kTile, false, vb > 0);
      mma_commit(&sh.mma);
    }
    // K and Q, where [dO; F] was
    if ((vb + 1 == blocks_v || !ok) && warp == 0 && elect_one()) {
      bar_arrive_tx(&sh.kq, kq_bytes(DK, NT));
      bulk_load(rb, kq + (ci * a.kheads + hk) * (long long)kq_bytes(DK, NT), kq_bytes(DK, NT),
                &sh.kq);
    }
    __syncwarp();
    ok = ok && wait_or_fail(&sh.mma, ph, failed, status);
    ph ^= 1;
    ok = __syncthreads_and(ok);
  }
  if (!ok && tid == 0) bar_wait(&sh.kq, 0);  // given up: no copy may land after the block has gone
  const int quarter = warp & 3, group = warp >> 2, lrow = quarter * 32 + lane;
  const uint32_t lb = tm + ((uint32_t)(quarter * 32) << 16) + group * 16;
  if (ok) {
    tc_fence_after();
    // X (rows 0 .. 63) and Z (64 .. 127) of [dO; F] E^T: this thread's row and 16
    // columns, each twice: times 2^ek_j for the products summed over j, times
    // 2^eq_i or 2^ek_i for those summed over i.
    const int i = lrow & 63;
    const bool is_z = lrow >= 64;
    uint32_t r[16];
    tmem_ld(lb + kColG, r);
    tmem_wait_ld();
    float x1[16], x2[16], m1 = 0.0f, m2 = 0.0f;
    const float inv = sh.of[lrow], bi = sh.beta[i], over = is_z ? sh.ek[i] : sh.eq[i];
    const float2 gi = sh.G[i];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int j = group * 16 + k;
      const float g = __uint_as_float(r[k]) * inv * sh.e[j];
      if (is_z && j == i && i < c.n)
        ga.dbeta[(packed ? c.row + i : c.b * a.tokens + c.row + i) * a.vheads + h] = g;
      float x = 0.0f;
      if (is_z ? j < i : j <= i)
        x = decay_between(gi, sh.G[j]) * sh.beta[j] * g * (is_z ? -bi : a.scale);
      x1[k] = x * sh.ek[j];
      x2[k] = x * over;
      m1 = fmaxf(m1, fabsf(x1[k]));
      m2 = fmaxf(m2, fabsf(x2[k]));
    }
    m1 = lane_max<32>(m1);
    m2 = lane_max<32>(m2);
    if (lane == 0) {  // (of values that are not negative the bits are in order)
      atomicMax(&sh.most[is_z ? 1 : 0], __float_as_uint(m1));
      atomicMax(&sh.most[2], __float_as_uint(m2));
    }
    __syncthreads();
    const float s1 = bound_scale(__uint_as_float(sh.most[is_z ? 1 : 0]));
    const float s2 = bound_scale(__uint_as_float(sh.most[2]));
    // Tiles in place of dS: X1, X2, Z1, Z2, two parts each.
    char *tiles = ra + (is_z ? 4 * kTile : 0);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float f[8], g[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        f[k] = x1[8 * p + k];
        g[k] = x2[8 * p + k];
      }
      uint4 hi, lo;
      const int at = piece_at(i, group * 2 + p, 0);
      split8(f, s1, hi, lo);
      *reinterpret_cast<uint4 *>(tiles + at) = hi;
      *reinterpret_cast<uint4 *>(tiles + kTile + at) = lo;
      split8(g, s2, hi, lo);
      *reinterpret_cast<uint4 *>(tiles + 2 * kTile + at) = hi;
      *reinterpret_cast<uint4 *>(tiles + 3 * kTile + at) = lo;
    }
    fence_smem_to_async();
    ok = wait_or_fail(&sh.kq, 0, failed, status);
    tc_fence_before();
    ok = __syncthreads_and(ok);
    tc_fence_after();
  }
  if (ok) {
    if (warp == 0 && elect_one()) {
      mma_tokens<DK, NT, false>(tm + kColQ2, sb, sa, false);
      mma_tokens<DK, NT, false>(tm + kColR2, sb, sa + 4 * kTile, false);
      mma_tokens<DK, NT, true>(tm + kColW2, sb + kTile, sa + 2 * kTile, false);
      mma_tokens<DK, NT, true>(tm + kColW2, sb, sa + 6 * kTile, true);
      mma_commit(&sh.mma);
    }
    __syncwarp();
    ok = wait_or_fail(&sh.mma, ph, failed, status);
  }
  if (__syncthreads_and(ok)) {
    tc_fence_after();
    const float ix = scale_inverse(bound_scale(__uint_as_float(sh.most[0])));
    const float iz = scale_inverse(bound_scale(__uint_as_float(sh.most[1])));
    const float iw = scale_inverse(bound_scale(__uint_as_float(sh.most[2])));
    // Row lrow of dk (columns of K), 16 tokens.
    const bool live = lrow < a.dk;
    const float is = lrow < DK ? sh.s0[lrow] : 0.0f, ids = lrow < DK ? sh.ds[lrow] : 0.0f;
    uint32_t r[16];
    float dot[16], w[16], out[16];
    float k_w = 0.0f;  // sum_j k_j . (Gamma/gamma beta dS E)_j
    auto element = [&](int tok, int which) {  // of K (0) or Q (1)
      const char *p = rb + which * kTile + (lrow >> 6) * 2 * kTile + tok * 128 +
                      ((((lrow >> 3) & 7) ^ (tok & 7)) << 4) + (lrow & 7) * 2;
      float x = __half2float(*reinterpret_cast<const __half *>(p));
      if constexpr (NT == 2)
        x += __half2float(*reinterpret_cast<const __half *>(p + 2 * (DK / 64) * kTile));
      return live ? x * (which ? sh.eq[tok] : sh.ek[tok]) : 0.0f;
    };
    auto put = [&](void *dst, int which, const float (&v)[16]) {
      if (!live) return;
      if constexpr (PARTIAL) {
        float *p = (which ? fs : es) + slot * (64 * 128) + lrow;
#pragma unroll
        for (int k = 0; k < 16; ++k) p[(group * 16 + k) * DK] = v[k];
      } else {
        const long long row = packed ? c.row : c.b * a.tokens + c.row;
        T *p = static_cast<T *>(dst) + (row * a.kheads + hk) * a.dk + lrow;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int t = group * 16 + k;
          if (t < c.n) p[(long long)t * a.kheads * a.dk] = from_acc<T>(v[k]);
        }
      }
    };
    // dQ
    tmem_ld(lb + kColQ1, r);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int t = group * 16 + k;
      out[k] = __uint_as_float(r[k]) * (is * sh.of[t] * sh.gam[t] * a.scale);
    }
    tmem_ld(lb + kColQ2, r);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      out[k] = fmaf(__uint_as_float(r[k]), ix, out[k]);
      dot[k] = element(group * 16 + k, 1) * out[k];
    }
    put(ga.dq, 0, out);
    // dKw
    tmem_ld(lb + kColW1, r);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int t = group * 16 + k;
      w[k] = __uint_as_float(r[k]) * (ids * sh.e[t] * sh.dec[t] * sh.beta[t]);
      k_w = fmaf(element(t, 0), w[k], k_w);
    }
    tmem_ld(lb + kColW2, r);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) w[k] = fmaf(__uint_as_float(r[k]), iw, w[k]);
    // dKr
    tmem_ld(lb + kColR1, r);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int t = group * 16 + k;
      out[k] = __uint_as_float(r[k]) * (-is * sh.of[64 + t] * sh.gam[t] * sh.beta[t]);
    }
    tmem_ld(lb + kColR2, r);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      out[k] = fmaf(__uint_as_float(r[k]), iz, out[k]);
      dot[k] = fmaf(element(group * 16 + k, 0), out[k] - w[k], dot[k]);
      out[k] += w[k];
      if (!live) dot[k] = 0.0f;
    }
    put(ga.dk, 1, out);
    if (!live) k_w = 0.0f;
    // Sums over dk, and of <S0, dS> and k_w over the block.
    const float d = warp_sums(dot, lane);
    if ((lane & 1) == 0) sh.dots[quarter][group * 16 + (lane >> 1)] = d;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      inner += __shfl_xor_sync(0xffffffffu, inner, o);
      k_w += __shfl_xor_sync(0xffffffffu, k_w, o);
    }
    if (lane == 0) {
      sh.part[0][warp] = inner;
      sh.part[1][warp] = k_w;
    }
    __syncthreads();
    if (warp == 0) {
      float end = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) end += sh.part[1][k];
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) s += sh.part[0][k];
      end = fmaf(sh.gam[63], s, end);
      // sums from each token to the last: two tokens per lane
      auto dg = [&](int t) {
        return (sh.dots[0][t] + sh.dots[1][t]) + (sh.dots[2][t] + sh.dots[3][t]);
      };
      const float hi = dg(2 * lane + 1), lo = dg(2 * lane);
      float sum = hi + lo;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float t = __shfl_down_sync(0xffffffffu, sum, o);
        if (lane + o < 32) sum += t;
      }
      const float after = sum - (hi + lo);
      const long long row = packed ? c.row : c.b * a.tokens + c.row;
      float *p = ga.dg + row * a.vheads + h;
      if (2 * lane < c.n) p[2ll * lane * a.vheads] = sum + end;
      if (2 * lane + 1 < c.n) p[(2ll * lane + 1) * a.vheads] = after + hi + end;
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 0) tmem_free(tm, 512);
}

// dq and dk of the key heads from their value heads' partial sums.
template <typename T, int DK>
__global__ void __launch_bounds__(256)
delta_grad_sum_kernel(const DeltaArgs a, const DeltaGradArgs ga, const DeltaPlan plan,
                      const float *dq, const float *dk) {
  const int hk = blockIdx.x % a.kheads, group = a.vheads / a.kheads;
  const long long ci = blockIdx.x / a.kheads;
  DeltaChunk c;
  if (!delta_chunk(a, plan, ci, c)) return;
  const int blocks_v = (a.dv + 127) / 128;
  const float *src = blockIdx.y ? dk : dq;
  const long long row = plan.chunk0 ? c.row : c.b * a.tokens + c.row;
  T *dst = static_cast<T *>(blockIdx.y ? ga.dk : ga.dq) + (row * a.kheads + hk) * a.dk;
  for (int i = threadIdx.x; i < c.n * DK; i += 256) {
    const int t = i / DK, e = i % DK;
    if (e >= a.dk) continue;
    float s = 0.0f;
    for (int k = 0; k < group; ++k)
      s += src[(ci * a.vheads + hk * group + k) * blocks_v * (64 * 128) + i];
    dst[(long long)t * a.kheads * a.dk + e] = from_acc<T>(s);
  }
}

}  // namespace fftgb
