// delta_back.cuh -- the gated delta rule's gradients from chunk to chunk, last
// chunk first (delta.cuh): the mirror image of delta_scan.cuh.
//
// The state is dS^T, the gradient of the state that leaves the chunk (columns
// of v along the lanes, dk along the columns).  Per chunk
//   P = dS^T K^T, X = dO^T M;  dU = P Gamma/gamma + scale X;
//   F = dU T (T = (I + beta A)^-1);  dV = beta F;
//   dS^T <- dS^T Gamma - (gamma beta F) K + (scale gamma dO) Q.
// The chain is P -> dU -> F -> dS; X, the outputs and all loads run beside it.
// Roles, scales and bounds as there.  Left for the kernel that follows: dS of
// every chunk and F.
//
// Tensor memory (512 columns):
//   D (fp32)         0 .. DK - 1
//   dS (two fp16)             128, 192        P, then F   256 .. 319
//   dU, then gamma beta F     320, 352        X           448 .. 511
//   dO, then scale gamma dO   384, 416
#pragma once

#include "delta_scan.cuh"

namespace fftgb {

template <typename T, int DK, bool STAGED>
__device__ __forceinline__ void delta_back(const DeltaArgs &a, const DeltaGradArgs &ga,
                                           const DeltaPlan &plan, unsigned block, const char *kq,
                                           const char *images, char *dstates, char *fs, char *os_,
                                           float *scales, int *status) {
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
  const bool packed = plan.chunk0 != nullptr;
  char *stages = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  if (tid < 4 * kTops) bounds.top[tid / kTops][tid % kTops] = 0;
  const uint32_t tm = scan_begin(bars, &tmem_slot, &failed, STAGED, tid, warp);
  char *ring = stages + ST * kStage + (STAGED ? kRows16 : 0);
  auto wait = [&](uint64_t *b, uint32_t parity) { return wait_or_fail(b, parity, &failed, status); };
  const T *dout = static_cast<const T *>(ga.dout) + out_row(a, sp.b, sp.row0, packed, h);
  const long long ostep = (long long)a.vheads * a.dv;

  if (warp >= kScanWarps + 2) {
    if constexpr (STAGED)
      scan_store<T>(a, sp, packed, h, true, ga.dv, vb * 128, stages + ST * kStage, &bars, &failed,
                    status, warp - kScanWarps - 2, lane);
  } else if (warp == kScanWarps + 1) {
    scan_load<T, DK, STAGED>(a, sp, h, true, kq, images, dout + vb * 128, ostep, vb * 128, stages,
                             ring, &bars, &failed, status, lane);
  } else if (warp == kScanWarps) {
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
      if (!wait(&bars.of, ph)) break;  // dO is there
      tc_fence_after();
      if (elect_one()) {
        mma_inner<NT == 1>(tm + kColN, tm + kColWh, tm + kColWl, image + 2 * kTile, false);
        mma_commit(&bars.n);
      }
      __syncwarp();
      if (!wait(&bars.y, ph)) break;
      tc_fence_after();
      if (elect_one()) {
        mma_inner<>(tm + kColP, tm + kColYh, tm + kColYl, image, false);
        mma_commit(&bars.e);
      }
      __syncwarp();
      if (!wait(&bars.u, ph)) break;
      tc_fence_after();
      if (elect_one())
        mma_update<DK, NT>(tm + kColD, tm + kColWh, tm + kColWl, q, false);
      __syncwarp();
      if (!wait(&bars.w, ph)) break;
      tc_fence_after();
      if (elect_one()) {
        mma_update<DK, NT>(tm + kColD, tm + kColYh, tm + kColYl, k, true);
        mma_commit(&bars.s);
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
    constexpr int TK = kScanTok, SC = DK / kScanGroups, SP = SC / 16;
    const long long sat = ((sp.b * a.vheads + h) * a.dk) * (long long)a.dv + dvr;
    RowAgree agree{box, row, group, warp & 3, 0};
    auto chunk_of = [&](int it) { return sp.chunks - 1 - it; };
    auto saved = [&](long long c) { return ((sp.chunk0 + c) * a.vheads + h) * blocks_v + vb; };
    auto gates_of = [&](int it) {
      return reinterpret_cast<const float *>(ring + (it % kGateRing) * kGateBytes);
    };
    T vr[STAGED ? 1 : TK];
    const T *col = dout + (live ? dvr : a.dv - 1);
    auto fetch = [&](int it) {
      if constexpr (!STAGED) {
        const long long r0 = (long long)chunk_of(it) * kChunk;
        const int last = (int)(sp.rows - r0 < kChunk ? sp.rows - r0 : kChunk) - 1;
#pragma unroll
        for (int j = 0; j < TK; ++j) {
          const int t = group * TK + j < last ? group * TK + j : last;
          vr[j] = col[(r0 + t) * ostep];
        }
      }
    };
    float2 S[SP][8];
    float ss = 1.0f;
    auto put_state = [&](int it) {
      const long long c = chunk_of(it);
#pragma unroll
      for (int p = 0; p < SP; ++p) {
        const int at = group * SC + p * 16;
        put_split(lb + kColSh + at / 2, lb + kColSl + at / 2, S[p]);
      }
      tmem_wait_st();
      warp_arrive(&bars.sb, lane);
      const float xs = bounds.scale(it - 1, 1), by = scale_inverse(ss) * xs;
#pragma unroll
      for (int p = 0; p < SP; ++p) {
        float2 f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = mul2(S[p][j], both(by));
        put_slab<true>(dstates + saved(c) * (512 * DK), DK, 2, group * SC + p * 16, row, f, live);
      }
      if (tid == 0) scales[saved(c) * kScales + kScaleD] = scale_inverse(xs);
    };
    auto state_max = [&]() {
      float m = 0.0f;
#pragma unroll
      for (int p = 0; p < SP; ++p) m = max16(m, S[p]);
      return m;
    };
    auto initial = [&](int c) {
      return ga.dfinal && live && c < a.dk ? ga.dfinal[sat + (long long)c * a.dv] : 0.0f;
    };
#pragma unroll
    for (int p = 0; p < SP; ++p)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = group * SC + p * 16 + 2 * j;
        S[p][j] = make_float2(initial(c), initial(c + 1));
      }
    // dO of the chunk of step `it`.
    auto take = [&](int it, float2 (&f)[8]) {
      const T *xs = reinterpret_cast<const T *>(stages + (it % ST) * kStage + kStage - kRows16) +
                    group * TK * 128 + row;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f[j] = STAGED ? make_float2(to_acc(xs[2 * j * 128]), to_acc(xs[(2 * j + 1) * 128]))
                      : make_float2(to_acc(vr[STAGED ? 0 : 2 * j]),
                                    to_acc(vr[STAGED ? 0 : 2 * j + 1]));
    };
    bool ok = true;
    if (sp.chunks > 0) {
      fetch(0);
      const float smax = agree.largest(state_max(), 0.0f).x;
      ss = bound_scale(smax);
      bounds.enter(-1, 1, live ? smax : 0.0f, lane);
      asm volatile("bar.sync 5, %0;" ::"n"(kScanWarps * 32) : "memory");
#pragma unroll
      for (int p = 0; p < SP; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) S[p][j] = mul2(S[p][j], both(ss));
      put_state(0);
    }
    for (int it = 0; it < sp.chunks && ok; ++it) {
      const uint32_t ph = it & 1;
      const int c = chunk_of(it);
      const float *gates = gates_of(it) + group * TK;
      const float *chunk = gates_of(it) + kChunkAt;
      uint32_t r[16];
      float2 x[8];
      // While P is computed: the scales, and dO as an operand.
      if (!(ok = wait(&bars.full[it % ST], (it / ST) & 1))) break;
      take(it, x);
      const float2 most = agree.largest(state_max(), max16(0.0f, x));
      const float Gamma = chunk[0], inv_s = scale_inverse(ss), smax = most.x * inv_s;
      const float os = bound_scale(most.y);
      const float bx = chunk[2] * most.y;
      const float bw = fmaxf(fmaf(chunk[7], smax, chunk[4] * bx), chunk[5] * most.y);
      const float yb = fmaxf(fmaf(chunk[1], smax, bx), fmaxf(smax, most.y) * kApart);
      const float ys = bound_scale(yb);
      const float ws =
          bound_scale(fmaxf(bw, fmaxf(yb * fmaxf(1.0f, chunk[4]), chunk[5]) * kApart));
      const float inv_y = scale_inverse(ys);
      const float bs = fmaf(Gamma, smax, 256.0f * bw), next_ss = bound_scale(bs);
      bounds.enter(it, 0, live ? fmaf(chunk[6], smax, chunk[3] * bx) : 0.0f, lane);
      bounds.enter(it, 1, live ? bs : 0.0f, lane);
      bounds.enter(it, 2, live ? most.y : 0.0f, lane);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = mul2(x[j], both(os));
      if constexpr (NT == 1) put_lead(lb + kColWh + group * 8, x);
      else put_split(lb + kColWh + group * 8, lb + kColWl + group * 8, x);
      tmem_wait_st();
      warp_arrive(&bars.of, lane);
      // dU
      if (!(ok = wait(&bars.p, ph) && wait(&bars.n, ph))) break;
      tc_fence_after();
      tmem_ld(lb + kColN + group * TK, r);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[j] = mul2(pair(r, j), mul2(gate(gates + 64, j), both(scale_inverse(os) * ys)));
      tmem_ld(lb + kColP + group * TK, r);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[j] = fma2(mul2(gate(gates, j), both(inv_s * ys)), pair(r, j), x[j]);
      put_split(lb + kColYh + group * 8, lb + kColYl + group * 8, x);
      tmem_wait_st();
      warp_arrive(&bars.y, lane);
      // While F is computed: scale gamma dO, where dO was.
      take(it, x);
      const float fscale = bounds.scale(it, 0), oscale = bounds.scale(it, 2);
      {
        float2 f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = mul2(x[j], both(oscale));
        put_slab<NT == 2>(os_ + saved(c) * (64 * 128 * 2 * NT), 64, NT, group * TK, row, f, live);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = mul2(x[j], mul2(gate(gates + 5 * 64, j), both(ws)));
      put_split(lb + kColWh + group * 8, lb + kColWl + group * 8, x);
      tmem_wait_st();
      warp_arrive(&bars.u, lane);
      if (lane == 0) bar_arrive(&bars.empty[it % ST]);
      // gamma beta F, where dU was
      if (!(ok = wait(&bars.e, ph))) break;
      tc_fence_after();
      tmem_ld(lb + kColP + group * TK, r);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[j] = mul2(pair(r, j), mul2(gate(gates + 4 * 64, j), both(inv_y * ws)));
      put_split(lb + kColYh + group * 8, lb + kColYl + group * 8, x);
      tmem_wait_st();
      warp_arrive(&bars.w, lane);
      // While the new dS is computed: F itself (taken from tensor memory once
      // more, which saves registers), and dV = beta F
      tmem_ld(lb + kColP + group * TK, r);
      tmem_wait_ld();
      TokenValues<T> dv;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 y = mul2(pair(r, j), mul2(gate(gates + 2 * 64, j), both(inv_y)));
        dv.set(j, mul2(y, gate(gates + 3 * 64, j)));
        x[j] = mul2(y, both(fscale));
      }
      put_slab<true>(fs + saved(c) * (64 * 128 * 4), 64, 2, group * TK, row, x, live);
      if (tid == 0) {
        float *to = scales + saved(c) * kScales;
        to[kScaleF] = scale_inverse(fscale);
        to[kScaleO] = scale_inverse(oscale);
        bounds.clear(it);
      }
      if (STAGED) {
        if (it > 0 && !(ok = wait(&bars.got, ph ^ 1))) break;
        dv.put(stages + ST * kStage, group * TK, row, lane);
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.put);
      } else if (live) {
        const long long r0 = (long long)c * kChunk + group * TK;
        const long long left = sp.rows - r0;
        T *out = static_cast<T *>(ga.dv) + out_row(a, sp.b, sp.row0 + r0, packed, h) + dvr;
#pragma unroll
        for (int j = 0; j < TK; ++j)
          if (j < left) out[j * ostep] = dv.get(j);
      }
      const bool more = it + 1 < sp.chunks;
      if (more) fetch(it + 1);
      // The gradient of the state before
      const float keep = Gamma * inv_s * next_ss, add = scale_inverse(ws) * next_ss;
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
    if (ok && ga.dinitial && live) {
      const float inv = scale_inverse(ss);
#pragma unroll
      for (int p = 0; p < SP; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int c = group * SC + p * 16 + 2 * j;
          if (c < a.dk) ga.dinitial[sat + (long long)c * a.dv] = S[p][j].x * inv;
          if (c + 1 < a.dk) ga.dinitial[sat + (long long)(c + 1) * a.dv] = S[p][j].y * inv;
        }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kScanWarps) tmem_free(tm, 512);
}

// Both scans of the gradients in one launch: neither needs anything of the
// other, and each has one block per sequence, head and 128 columns of v, so
// apart they left most of the SMs idle (4 sequences of 4096 tokens, 16 heads of
// 128 x 128, 64 blocks each: 246 + 295 us; together 354, with HBM 57% busy by
// what they leave).  Even blocks go forwards, odd ones backwards.
template <typename T, int DK, bool STAGED>
__global__ void __launch_bounds__(kScanThreads, 1)
delta_scans_kernel(const DeltaArgs a, const DeltaGradArgs ga, const DeltaPlan plan, const char *kq,
                   const char *images, const char *back, char *states, char *dstates, char *es,
                   char *fs, char *os, float *scales, int *status) {
  if (blockIdx.x & 1)
    delta_back<T, DK, STAGED>(a, ga, plan, blockIdx.x >> 1, kq, back, dstates, fs, os, scales,
                              status);
  else
    delta_scan<T, DK, true, STAGED>(a, plan, blockIdx.x >> 1, kq, images, states, es, scales,
                                    status);
}

}  // namespace fftgb
