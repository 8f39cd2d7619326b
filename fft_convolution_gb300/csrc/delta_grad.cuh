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
// The products run transposed (dk along the lanes of tensor memory, tokens along
// the columns).  S0, dS, E, F and dO come as the scans left them, slabs of 16
// columns of v that are operands as they are: over a ring of slabs go
//   S0 [dO; F]^T (128 columns: dQ's and dKr's first parts), dS E^T, [dO; F] E^T,
// leading parts and trailing ones into accumulators of their own (the
// accumulator cuts off below its last bit at every step: with both in one,
// dbeta was 2.5 times as far off).  X and Z, from the last of them, become
// right operands of the products with K and Q.  Heads that share a key head
// leave fp32 partial sums, added by a small kernel in a fixed order.
//
// One block per SM walks over chunks and value heads: 16 warps turn
// accumulators into X, Z and the results; one thread issues the products; a
// warp copies slabs ahead, so that the next chunk's arrive while this one's
// results are written; two take <S0, dS> from the slabs.
//
// Each chunk and head reads 208 KB (128 x 128 heads of 16 bits) and its 16 warps
// then work 13000 clocks on 64 x 64 and 128 x 64 accumulators, a fifth of them
// waiting; HBM would need 9000.  16384 tokens of 16 heads: 258 us, 4.4 TB/s (as
// a block per chunk that loaded and split fp32 rows itself 675).  Of its 96
// registers per thread 16-bit types spill 44 bytes, 240 with more than 128 columns
// of v (fp32 16 and 208).
#pragma once

#include "delta_prep.cuh"
#include "delta_scan.cuh"

namespace fftgb {

constexpr int kGradWarps = 16, kGradThreads = (kGradWarps + 4) * 32;
// A slab: S0, dS and E (two parts each), [dO; F] leading, [dO; F] trailing.
__host__ __device__ constexpr int slab_e(int dk) { return 4 * slab_part(dk); }
__host__ __device__ constexpr int slab_of(int dk) { return slab_e(dk) + 2 * slab_part(64); }
__host__ __device__ constexpr int slab_bytes(int dk) { return slab_of(dk) + 2 * slab_part(128); }
__host__ __device__ constexpr int grad_slabs(int terms) { return terms == 1 ? 4 : 3; }
// K and Q; X and Z (two tiles of two parts each); the ring.
__host__ __device__ constexpr size_t grad_smem(int dk, int terms) {
  return 1024 + kq_bytes(dk, terms) + 8 * kTile + (size_t)grad_slabs(terms) * slab_bytes(dk);
}

struct alignas(16) GradTokens {
  float2 G[64];
  float beta[64], ek[64], eq[64];
  float fq[64], fr[64], fw[64];  // scale gamma, -gamma beta, Gamma/gamma beta; 0 past the chunk's end
  float Gamma;
  unsigned most[3];  // largest X1, Z1, and X2 or Z2
};
// Four tokens' factors.
__device__ __forceinline__ void four(const float *p, float (&f)[4]) {
  const float4 x = *reinterpret_cast<const float4 *>(p);
  f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
}
struct GradShared {
  uint64_t full[4], empty[4];       // slabs
  uint64_t kq, kq_free;             // K and Q there; read
  uint64_t first, tiles, second;    // products over v done; X and Z there; their products done
  uint64_t read;                    // accumulators read
  uint64_t inner, done;
  uint32_t tmem_slot;
  int failed;
  GradTokens tok[2];                // of this chunk and the next
  float inner_part[2][2];           // <S0, dS>
  float dots[4][64];
  float k_w[kGradWarps];
};

// A barrier of the 16 warps: whether `p` holds in all of their threads.
__device__ __forceinline__ bool grad_all(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "n"(kGradWarps * 32)
      : "memory");
  return r != 0;
}

// Between a warp's reads of shared memory and the arrival that lets a bulk copy
// overwrite it: without the fence the arrival overtook loads under way (<S0, dS>
// then summed values of the next slab, in 1 to 100% of calls).
__device__ __forceinline__ void read_before_copy() {
  __threadfence_block();
  fence_smem_to_async();
}

// D (128 lanes x N) (+)= A B^T over one slab.
template <int N>
__device__ __forceinline__ void mma_slab(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
  mma_ss_plain(d, a, b, mma_desc(128, N, true, true), accumulate);
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

// Columns of tensor memory: leading and trailing accumulators of S0 [dO; F]^T,
// dS E^T and [dO; F] E^T; later, in place of the last two, the products with K
// and Q.
constexpr uint32_t kAccQ = 0, kAccQt = 128, kAccW = 256, kAccWt = 320, kAccG = 384, kAccGt = 448;

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

// A thread's column of dk of 16 tokens, `step` apart.  Two lanes exchange every
// other token, so that each stores two columns at once (PAIRS).
template <typename T, bool PAIRS>
__device__ __forceinline__ void put_tokens(T *p, long long step, int tokens, bool live, int lane,
                                           const float (&v)[16]) {
  if constexpr (PAIRS) {
    const int odd = lane & 1;
    uint32_t *w = reinterpret_cast<uint32_t *>(p - odd + odd * step);
    float x[16];
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const float o = __shfl_xor_sync(0xffffffffu, odd ? v[k] : v[k + 1], 1);
      x[k] = odd ? o : v[k];
      x[k + 1] = odd ? v[k + 1] : o;
    }
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      T pair[2] = {from_acc<T>(x[k]), from_acc<T>(x[k + 1])};
      if (live && k + odd < tokens) *w = *reinterpret_cast<const uint32_t *>(pair);
      w = reinterpret_cast<uint32_t *>(reinterpret_cast<T *>(w) + 2 * step);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (live && k < tokens) *p = from_acc<T>(v[k]);
      p += step;
    }
  }
}

// partial: dq and dk of this value head go to fp32 arrays [64][DK] in place of
// the chunk's E and F, which only this block reads, else to their arrays.
// MULTI: more than 128 columns of v, whose sums are kept in registers; with one
// block of columns they stay in tensor memory until X and Z are done (kept in
// registers they spilled, and the little memory beside the ring is no cache:
// 424 us against 250).
template <typename T, int DK, bool MULTI>
__global__ void __launch_bounds__(kGradThreads, 1)
delta_grad_kernel(const DeltaArgs a, const DeltaGradArgs ga, const DeltaPlan plan, const char *kq,
                  const char *back, const char *states, const char *dstates, char *es, char *fs,
                  const char *os, const float *scales, bool partial, int *status) {
  extern __shared__ char smem_raw[];
  __shared__ GradShared sh;
  constexpr int NT = Terms<T>::value, R = grad_slabs(NT), kSlabBytes = slab_bytes(DK);
  constexpr int kE = slab_e(DK), kOF = slab_of(DK), kPart = slab_part(64);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  char *ra = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  char *rb = ra + 8 * kTile, *ring = rb + kq_bytes(DK, NT);
  const int blocks_v = MULTI ? (a.dv + 127) / 128 : 1;
  const bool packed = plan.chunk0 != nullptr;
  const long long items = (packed ? (long long)plan.chunk0[a.batch] : plan.chunks_max) * a.vheads;
  volatile int *failed = &sh.failed;
  auto wait = [&](uint64_t *b, uint32_t parity) { return wait_or_fail(b, parity, failed, status); };

  if (warp == kGradWarps) tmem_alloc(&sh.tmem_slot, 512);
  if (tid == 0) {
    for (int s = 0; s < R; ++s) {
      bar_init(&sh.full[s], 1);
      bar_init(&sh.empty[s], 3);
    }
    for (uint64_t *b : {&sh.kq, &sh.first, &sh.second, &sh.done}) bar_init(b, 1);
    for (uint64_t *b : {&sh.kq_free, &sh.tiles, &sh.read}) bar_init(b, kGradWarps);
    bar_init(&sh.inner, 2);
    sh.failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (NT == 1) {  // one value holds dO: its trailing part stays 0
    for (int i = tid; i < R * (kPart / 16); i += kGradThreads)
      *reinterpret_cast<uint4 *>(ring + (i / (kPart / 16)) * kSlabBytes + kOF + 2 * kPart +
                                 (i % (kPart / 16)) * 16) = make_uint4(0, 0, 0, 0);
    fence_smem_to_async();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, sh.tmem_slot, 0);

  if (warp == kGradWarps + 1) {
    // Copies: K and Q after the first slabs, since they wait for the chunk before.
    if (elect_one()) {
      long long n = 0, kqs = 0;
      bool ok = true;
      for (long long i = blockIdx.x; i < items && ok; i += gridDim.x) {
        const long long ci = i / a.vheads;
        const int h = (int)(i % a.vheads), hk = h / (a.vheads / a.kheads);
        for (int k = 0; k < blocks_v * kSlabs && ok; ++k, ++n) {
          if (k == R) {
            if (!(ok = kqs == 0 || wait(&sh.kq_free, (kqs - 1) & 1))) break;
            bar_arrive_tx(&sh.kq, kq_bytes(DK, NT));
            bulk_load(rb, kq + (ci * a.kheads + hk) * (long long)kq_bytes(DK, NT),
                      kq_bytes(DK, NT), &sh.kq);
            ++kqs;
          }
          const int s = (int)(n % R);
          if (!(ok = n < R || wait(&sh.empty[s], (n / R - 1) & 1))) break;
          const long long slot = i * blocks_v + (k >> 3);
          const int sl = k & 7;
          char *dst = ring + s * kSlabBytes;
          uint64_t *bar = &sh.full[s];
          bar_arrive_tx(bar, 4 * slab_part(DK) + 4 * kPart + NT * kPart);
          bulk_load(dst, states + slot * (512 * DK) + sl * 2 * slab_part(DK), 2 * slab_part(DK), bar);
          bulk_load(dst + 2 * slab_part(DK), dstates + slot * (512 * DK) + sl * 2 * slab_part(DK),
                    2 * slab_part(DK), bar);
          bulk_load(dst + kE, es + slot * (kSlabs * 2 * kPart) + sl * 2 * kPart, 2 * kPart, bar);
          const char *f = fs + slot * (kSlabs * 2 * kPart) + sl * 2 * kPart;
          const char *o = os + (slot * kSlabs + sl) * (NT * kPart);
          bulk_load(dst + kOF, o, kPart, bar);
          bulk_load(dst + kOF + kPart, f, kPart, bar);
          if (NT == 2) bulk_load(dst + kOF + 2 * kPart, o + kPart, kPart, bar);
          bulk_load(dst + kOF + 3 * kPart, f + kPart, kPart, bar);
        }
      }
      if (*failed) {  // given up: no copy may land after the block has gone
        for (long long k = n > R ? n - R : 0; k < n; ++k) bar_wait(&sh.full[k % R], (k / R) & 1);
        if (kqs > 0) bar_wait(&sh.kq, (kqs - 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == kGradWarps) {
    long long n = 0, phases = 0;
    uint32_t item = 0;
    bool ok = true;
    const uint32_t sa = smem_u32(ra), sb = smem_u32(rb), slabs = smem_u32(ring);
    for (long long i = blockIdx.x; i < items && ok; i += gridDim.x, ++item) {
      for (int vb = 0; vb < blocks_v && ok; ++vb, ++phases) {
        if (!(ok = phases == 0 || wait(&sh.read, (phases - 1) & 1))) break;
        for (int k = 0; k < kSlabs; ++k, ++n) {
          const int s = (int)(n % R);
          if (!(ok = wait(&sh.full[s], (n / R) & 1))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t S = slabs + s * kSlabBytes, D = S + 2 * slab_part(DK), E = S + kE,
                           OF = S + kOF;
            mma_slab<128>(tm + kAccQt, S + slab_part(DK), OF, k > 0);
            if (NT == 2) mma_slab<128>(tm + kAccQt, S, OF + 2 * kPart, true);
            else mma_slab<64>(tm + kAccQt + 64, S, OF + 3 * kPart, true);
            mma_slab<128>(tm + kAccQ, S, OF, k > 0);
            mma_slab<64>(tm + kAccWt, D + slab_part(DK), E, k > 0);
            mma_slab<64>(tm + kAccWt, D, E + kPart, true);
            mma_slab<64>(tm + kAccW, D, E, k > 0);
            mma_slab<64>(tm + kAccGt, OF + 2 * kPart, E, k > 0);
            mma_slab<64>(tm + kAccGt, OF, E + kPart, true);
            mma_slab<64>(tm + kAccG, OF, E, k > 0);
            mma_commit(&sh.empty[s]);
            if (k == kSlabs - 1) mma_commit(&sh.first);
          }
          __syncwarp();
        }
      }
      ok = ok && wait(&sh.tiles, item & 1) && wait(&sh.kq, item & 1);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        mma_tokens<DK, NT, false>(tm + kAccG, sb, sa, false);
        mma_tokens<DK, NT, false>(tm + kAccGt, sb, sa + 4 * kTile, false);
        mma_tokens<DK, NT, true>(tm + kAccW, sb + kTile, sa + 2 * kTile, false);
        mma_tokens<DK, NT, true>(tm + kAccW, sb, sa + 6 * kTile, true);
        mma_commit(&sh.second);
      }
      __syncwarp();
    }
    if (elect_one()) {
      mma_commit(&sh.done);
      bar_wait(&sh.done, 0);
    }
    __syncwarp();
  } else if (warp > kGradWarps) {
    // <S0, dS>, half of every slab's pieces of eight values each
    const int which = warp - kGradWarps - 2, piece = which * 32 + lane;
    long long n = 0;
    uint32_t item = 0;
    bool ok = true;
    for (long long i = blockIdx.x; i < items && ok; i += gridDim.x, ++item) {
      float inner = 0.0f;
      for (int vb = 0; vb < blocks_v && ok; ++vb) {
        const float *sc = scales + (i * blocks_v + vb) * kScales;
        const float is = sc[kScaleS], ids = sc[kScaleD];
        float sum = 0.0f;
        for (int k = 0; k < kSlabs; ++k, ++n) {
          const int s = (int)(n % R);
          if (!(ok = wait(&sh.full[s], (n / R) & 1))) break;
          const char *S = ring + s * kSlabBytes + piece * 16, *D = S + 2 * slab_part(DK);
#pragma unroll
          for (int j = 0; j < slab_part(DK) / (64 * 16); ++j) {
            const uint4 sh4 = *reinterpret_cast<const uint4 *>(S + j * 1024);
            const uint4 sl4 = *reinterpret_cast<const uint4 *>(S + j * 1024 + slab_part(DK));
            const uint4 dh4 = *reinterpret_cast<const uint4 *>(D + j * 1024);
            const uint4 dl4 = *reinterpret_cast<const uint4 *>(D + j * 1024 + slab_part(DK));
            auto both_parts = [](uint32_t h, uint32_t l) {
              const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h));
              const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&l));
              return make_float2(x.x + y.x, x.y + y.y);
            };
            auto add = [&](uint32_t h, uint32_t l, uint32_t dh, uint32_t dl) {
              const float2 x = both_parts(h, l), y = both_parts(dh, dl);
              sum = fmaf(x.x, y.x, fmaf(x.y, y.y, sum));
            };
            add(sh4.x, sl4.x, dh4.x, dl4.x);
            add(sh4.y, sl4.y, dh4.y, dl4.y);
            add(sh4.z, sl4.z, dh4.z, dl4.z);
            add(sh4.w, sl4.w, dh4.w, dl4.w);
          }
          read_before_copy();
          __syncwarp();
          if (lane == 0) bar_arrive(&sh.empty[s]);
        }
        inner = fmaf(sum * is, ids, inner);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, o);
      if (lane == 0) {
        sh.inner_part[item & 1][which] = inner;
        bar_arrive(&sh.inner);
      }
    }
  } else {
    const int quarter = warp & 3, group = warp >> 2, lrow = quarter * 32 + lane;
    const uint32_t lb = tm + ((uint32_t)(quarter * 32) << 16) + group * 16;
    const int i = lrow & 63;         // of [dO; F] E^T: token
    const bool is_z = lrow >= 64, live = lrow < a.dk;
    uint32_t item = 0, phases = 0;
    bool ok = true;
    for (long long it = blockIdx.x; it < items; it += gridDim.x, ++item) {
      const long long ci = it / a.vheads, slot = it * blocks_v;
      const int h = (int)(it % a.vheads), hk = h / (a.vheads / a.kheads);
      DeltaChunk c;
      delta_chunk(a, plan, ci, c);
      GradTokens &tk = sh.tok[item & 1];
      if (warp == 0) {
        running_decay_warp(a.g + c.b * a.sg.seq + c.row * a.sg.tok + h * a.sg.head, a.sg.tok, c.n,
                           lane, tk.G);
      } else if (warp == 1) {
        const float *gates = reinterpret_cast<const float *>(
            back + (ci * a.vheads + h) * (long long)kImageBytes + 4 * kTile);
#pragma unroll
        for (int t = lane; t < 64; t += 32) {
          tk.beta[t] = gates[3 * 64 + t];
          tk.ek[t] = gates[6 * 64 + t];
          tk.eq[t] = gates[7 * 64 + t];
        }
        if (lane < 3) tk.most[lane] = 0;
      }
      // The products over v
      float q1[16], r1[16], w1[16], gx[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) q1[k] = r1[k] = w1[k] = gx[k] = 0.0f;
      auto take = [&](uint32_t lead, uint32_t trail, float x, float y, float (&to)[16]) {
        uint32_t r[16], t[16];
        tmem_ld(lb + lead, r);
        tmem_ld(lb + trail, t);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k)
          to[k] = fmaf((__uint_as_float(r[k]) + __uint_as_float(t[k])) * x, y, to[k]);
      };
      float is = 0.0f, jf = 0.0f, jo = 0.0f;
      for (int vb = 0; vb < blocks_v; ++vb, ++phases) {
        const float *sc = scales + (slot + vb) * kScales;
        const float ie = sc[kScaleE], ids = sc[kScaleD];
        is = sc[kScaleS];
        jf = sc[kScaleF];
        jo = sc[kScaleO];
        ok = ok && wait(&sh.first, phases & 1);
        tc_fence_after();
        take(kAccG, kAccGt, is_z ? jf : jo, ie, gx);
        take(kAccW, kAccWt, ids, ie, w1);
        if (MULTI) {
          take(kAccQ, kAccQt, is, jo, q1);
          take(kAccQ + 64, kAccQt + 64, is, jf, r1);
          if (vb + 1 < blocks_v) warp_arrive(&sh.read, lane);
        }
      }
      ok = grad_all(ok);
      if (!ok) break;
      if (warp < 2) {
        const int t = tid;
        const float gam = decay_between(tk.G[t], make_float2(0.0f, 0.0f)), bt = tk.beta[t];
        const bool there = t < c.n;
        tk.fq[t] = there ? gam * a.scale : 0.0f;
        tk.fr[t] = there ? -gam * bt : 0.0f;
        tk.fw[t] = there ? decay_between(tk.G[63], tk.G[t]) * bt : 0.0f;
        if (t == 63) tk.Gamma = gam;
      }
      // X (rows 0 .. 63) and Z (64 .. 127) of [dO; F] E^T: this thread's row and 16
      // columns, each twice: times 2^ek_j for the products summed over j, times
      // 2^eq_i or 2^ek_i for those summed over i.
      {
        float m1 = 0.0f, m2 = 0.0f;
        const float bi = is_z ? -tk.beta[i] : a.scale, over = is_z ? tk.ek[i] : tk.eq[i];
        const float2 gi = tk.G[i];
        const int last = (i < c.n ? is_z ? i - 1 : i : -1) - group * 16;
        const int diagonal = is_z && i < c.n ? i - group * 16 : -1;
        float *db = ga.dbeta + (packed ? c.row + i : c.b * a.tokens + c.row + i) * a.vheads + h;
#pragma unroll
        for (int k0 = 0; k0 < 16; k0 += 4) {
          float bj[4], ej[4];
          four(tk.beta + group * 16 + k0, bj);
          four(tk.ek + group * 16 + k0, ej);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = k0 + e;
            if (k == diagonal) *db = gx[k];
            gx[k] = k <= last ? decay_between(gi, tk.G[group * 16 + k]) * bj[e] * gx[k] * bi : 0.0f;
            m1 = fmaxf(m1, fabsf(gx[k] * ej[e]));
            m2 = fmaxf(m2, fabsf(gx[k]));
          }
        }
        m1 = lane_max<32>(m1);
        m2 = lane_max<32>(m2 * over);
        if (lane == 0) {  // (of values that are not negative the bits are in order)
          atomicMax(&tk.most[is_z ? 1 : 0], __float_as_uint(m1));
          atomicMax(&tk.most[2], __float_as_uint(m2));
        }
        grad_all(true);
        const float s1 = bound_scale(__uint_as_float(tk.most[is_z ? 1 : 0]));
        const float s2 = bound_scale(__uint_as_float(tk.most[2]));
        char *tiles = ra + (is_z ? 4 * kTile : 0);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float f[8], g[8];
#pragma unroll
          for (int k = 0; k < 8; k += 4) {
            float ej[4];
            four(tk.ek + group * 16 + 8 * p + k, ej);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[k + e] = gx[8 * p + k + e] * ej[e];
              g[k + e] = gx[8 * p + k + e] * over;
            }
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
        warp_arrive(&sh.tiles, lane);
      }
      if (!MULTI) {
        take(kAccQ, kAccQt, is, jo, q1);
        take(kAccQ + 64, kAccQt + 64, is, jf, r1);
      }
      ok = wait(&sh.kq, item & 1);
      // Row lrow of dk of K (0) or Q (1), a token's value without its scale
      auto element = [&](int tok, int which) {
        const char *p = rb + which * kTile + (lrow >> 6) * 2 * kTile + tok * 128 +
                        ((((lrow >> 3) & 7) ^ (tok & 7)) << 4) + (lrow & 7) * 2;
        float x = __half2float(*reinterpret_cast<const __half *>(p));
        if constexpr (NT == 2)
          x += __half2float(*reinterpret_cast<const __half *>(p + 2 * (DK / 64) * kTile));
        return x;
      };
      float k_w = 0.0f, dot[16];  // k_w: sum_j k_j . (Gamma/gamma beta dS E)_j
#pragma unroll
      for (int k0 = 0; k0 < 16; k0 += 4) {
        float fq[4], fr[4], fw[4], ek[4];
        four(tk.fq + group * 16 + k0, fq);
        four(tk.fr + group * 16 + k0, fr);
        four(tk.fw + group * 16 + k0, fw);
        four(tk.ek + group * 16 + k0, ek);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = k0 + e;
          q1[k] *= fq[e];
          r1[k] *= fr[e];
          w1[k] *= fw[e];
          dot[k] = element(group * 16 + k, 0) * ek[e];
          k_w = fmaf(dot[k], w1[k], k_w);
        }
      }
      // The products over tokens
      ok = ok && wait(&sh.second, item & 1);
      tc_fence_after();
      {
        auto add = [&](uint32_t col, int which, float (&to)[16]) {
          const float x = scale_inverse(bound_scale(__uint_as_float(tk.most[which])));
          uint32_t r[16];
          tmem_ld(lb + col, r);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) to[k] = fmaf(__uint_as_float(r[k]), x, to[k]);
        };
        add(kAccG, 0, q1);
        add(kAccGt, 1, r1);
        add(kAccW, 2, w1);
      }
      ok = ok && wait(&sh.inner, item & 1);
      warp_arrive(&sh.read, lane);
      const int tokens = c.n - group * 16;  // of these 16
#pragma unroll
      for (int k0 = 0; k0 < 16; k0 += 4) {
        float eq[4];
        four(tk.eq + group * 16 + k0, eq);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = k0 + e;
          dot[k] = fmaf(dot[k], r1[k] - w1[k], element(group * 16 + k, 1) * eq[e] * q1[k]);
          if (!live || k >= tokens) dot[k] = 0.0f;
          r1[k] += w1[k];
        }
      }
      if (!live) k_w = 0.0f;
      const float d = warp_sums(dot, lane);
      read_before_copy();
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.kq_free);
      if ((lane & 1) == 0) sh.dots[quarter][group * 16 + (lane >> 1)] = d;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) k_w += __shfl_xor_sync(0xffffffffu, k_w, o);
      if (lane == 0) sh.k_w[warp] = k_w;
      if (partial) {
        const long long at = slot * (64 * 128) + group * 16 * DK + lrow;
        put_tokens<float, false>(reinterpret_cast<float *>(es) + at, DK, 16, lrow < DK, lane, q1);
        put_tokens<float, false>(reinterpret_cast<float *>(fs) + at, DK, 16, lrow < DK, lane, r1);
      } else {
        const long long step = (long long)a.kheads * a.dk;
        const long long row = (packed ? c.row : c.b * a.tokens + c.row) + group * 16;
        T *dq = static_cast<T *>(ga.dq) + row * step + hk * a.dk + lrow;
        T *dk = static_cast<T *>(ga.dk) + row * step + hk * a.dk + lrow;
        if (sizeof(T) == 2 && a.dk % 2 == 0 && (((uintptr_t)ga.dq | (uintptr_t)ga.dk) & 3u) == 0) {
          put_tokens<T, sizeof(T) == 2>(dq, step, tokens, live, lane, q1);
          put_tokens<T, sizeof(T) == 2>(dk, step, tokens, live, lane, r1);
        } else {
          put_tokens<T, false>(dq, step, tokens, live, lane, q1);
          put_tokens<T, false>(dk, step, tokens, live, lane, r1);
        }
      }
      ok = grad_all(ok);
      if (!ok) break;
      if (warp == 0) {
        float end = 0.0f;
#pragma unroll
        for (int k = 0; k < kGradWarps; ++k) end += sh.k_w[k];
        end = fmaf(tk.Gamma, sh.inner_part[item & 1][0] + sh.inner_part[item & 1][1], end);
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
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kGradWarps) tmem_free(tm, 512);
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
