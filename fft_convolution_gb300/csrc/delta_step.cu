// delta_step.cu -- the gated delta rule one token after the other, for
// decoding: a few tokens per sequence against a state that stays in HBM
// between calls.
//
// Per token  S <- e^g S;  u = beta (v - S^T k);  S <- S + k u^T;
//            o = scale S^T q.
// With S' the decayed state, S^T q = S'^T q + (k . q) u: both products with
// the state are taken in one walk over it, and one exchange between the
// threads gives every sum.  The state changes by k u + S (e^g - 1), added in
// one rounding: of a slow decay e^g itself would keep few digits of its
// distance from 1, an error that thousands of tokens add up; what rounding
// leaves out of u is carried along for the same reason.
//
// Reading and writing the fp32 state is nearly all the traffic (128 KB per
// head of 128 x 128, against under 1 KB for the token), so HBM bounds the
// kernel.  A block owns 32 columns of one head's state: their rows are whole
// 128-byte lines, a single sequence still spreads over dv / 32 blocks per
// head, and a block's share of the state fits the registers of 128 threads
// (4 columns and dk / 16 rows each), so the state is read once and written
// once however many tokens the call has.
#include "seq.h"

namespace fftgb {

constexpr int kStepThreads = 128, kStepCols = 32;

template <typename T, int R, bool VEC>
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(const DeltaArgs a) {
  __shared__ float red[2][4][8][9];
  const int tiles = (a.dv + kStepCols - 1) / kStepCols;
  const int tile = blockIdx.x % tiles;
  const long long bh = blockIdx.x / tiles;
  const int h = (int)(bh % a.vheads);
  const long long b = bh / a.vheads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cg = lane & 7;                 // 4 columns
  const int rg = warp * 4 + (lane >> 3);   // rows rg, rg + 16, ...
  const int c0 = tile * kStepCols + cg * 4;
  const int hk = h / (a.vheads / a.kheads);

  T *o = static_cast<T *>(a.o) + ((b * a.tokens) * a.vheads + h) * a.dv;
  const long long ostep = (long long)a.vheads * a.dv;
  const long long slot = a.slots ? a.slots[b] : b;
  if (slot < 0 || slot >= a.pool) {
    if (rg == 0)
      for (long long t = 0; t < a.tokens; ++t)
        for (int j = 0; j < 4; ++j)
          if (c0 + j < a.dv) o[t * ostep + c0 + j] = from_acc<T>(0.0f);
    return;
  }
  const long long at = (slot * a.vheads + h) * a.dk * a.dv;
  const float *sin = a.state_in ? a.state_in + at : nullptr;
  float *sout = a.state_out ? a.state_out + at : nullptr;

  float s[R][4];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = rg + 16 * i;
    if (sin && r < a.dk) {
      if constexpr (VEC) {
        float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c0 < a.dv) f = *reinterpret_cast<const float4 *>(sin + (long long)r * a.dv + c0);
        s[i][0] = f.x; s[i][1] = f.y; s[i][2] = f.z; s[i][3] = f.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = c0 + j < a.dv ? sin[(long long)r * a.dv + c0 + j] : 0.0f;
      }
    } else {
      s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
    }
  }

  const T *q = static_cast<const T *>(a.q) + b * a.sq.seq + hk * a.sq.head;
  const T *k = static_cast<const T *>(a.k) + b * a.sk.seq + hk * a.sk.head;
  const T *v = static_cast<const T *>(a.v) + b * a.sv.seq + h * a.sv.head;
  const float *g = a.g + b * a.sg.seq + h * a.sg.head;
  const float *beta = a.beta + b * a.sb.seq + h * a.sb.head;
  for (long long t = 0; t < a.tokens; ++t) {
    float kr[R], qr[R], vc[4];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = rg + 16 * i;
      kr[i] = r < a.dk ? to_acc(k[t * a.sk.tok + r]) : 0.0f;
      qr[i] = r < a.dk ? to_acc(q[t * a.sq.tok + r]) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) vc[j] = c0 + j < a.dv ? to_acc(v[t * a.sv.tok + c0 + j]) : 0.0f;
    const float decay = expm1f(g[t * a.sg.tok]), bt = beta[t * a.sb.tok];
    float sum[9];  // S^T k and S^T q of the 4 columns (S before its decay), k . q
#pragma unroll
    for (int j = 0; j < 9; ++j) sum[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum[j] = fmaf(kr[i], s[i][j], sum[j]);
        sum[4 + j] = fmaf(qr[i], s[i][j], sum[4 + j]);
      }
      sum[8] = fmaf(kr[i], qr[i], sum[8]);
    }
    float(*rd)[8][9] = red[t & 1];
#pragma unroll
    for (int j = 0; j < 9; ++j) {
      sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 8);
      sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 16);
      if (lane < 8) rd[warp][cg][j] = sum[j];
    }
    __syncthreads();  // the two halves of `red` alternate: one barrier per token
#pragma unroll
    for (int j = 0; j < 9; ++j)
      sum[j] = (rd[0][cg][j] + rd[1][cg][j]) + (rd[2][cg][j] + rd[3][cg][j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // u = beta (v - S'^T k) and what its rounding leaves out
      const float held = fmaf(decay, sum[j], sum[j]), miss = vc[j] - held;
      const float back = miss - vc[j];
      const float rest = (vc[j] - (miss - back)) - (held + back);
      const float u = bt * miss, ur = fmaf(bt, miss, -u) + bt * rest;
#pragma unroll
      for (int i = 0; i < R; ++i)
        s[i][j] += fmaf(kr[i], u, fmaf(kr[i], ur, decay * s[i][j]));
      if (rg == 0 && c0 + j < a.dv)
        o[t * ostep + c0 + j] =
            from_acc<T>(a.scale * fmaf(sum[8], u, fmaf(decay, sum[4 + j], sum[4 + j])));
    }
  }

  if (!sout) return;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = rg + 16 * i;
    if (r >= a.dk) continue;
    if constexpr (VEC) {
      if (c0 < a.dv)
        *reinterpret_cast<float4 *>(sout + (long long)r * a.dv + c0) =
            make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c0 + j < a.dv) sout[(long long)r * a.dv + c0 + j] = s[i][j];
    }
  }
}

template <typename T>
static cudaError_t delta_step_t(const DeltaArgs &a, cudaStream_t st) {
  const long long blocks = a.batch * a.vheads * ((a.dv + kStepCols - 1) / kStepCols);
  const bool vec = a.dv % 4 == 0 && (((uintptr_t)a.state_in | (uintptr_t)a.state_out) & 15u) == 0;
  auto run = [&](auto kern) {
    kern<<<(unsigned)blocks, kStepThreads, 0, st>>>(a);
    return cudaGetLastError();
  };
  if (a.dk <= 64) return vec ? run(delta_step_kernel<T, 4, true>) : run(delta_step_kernel<T, 4, false>);
  if (a.dk <= 128)
    return vec ? run(delta_step_kernel<T, 8, true>) : run(delta_step_kernel<T, 8, false>);
  return vec ? run(delta_step_kernel<T, 16, true>) : run(delta_step_kernel<T, 16, false>);
}

cudaError_t launch_delta_step(int dtype, const DeltaArgs &a, cudaStream_t st) {
  if (dtype == FFT_ELEM_F32) return delta_step_t<float>(a, st);
  if (dtype == FFT_ELEM_BF16) return delta_step_t<__nv_bfloat16>(a, st);
  return delta_step_t<__half>(a, st);
}

}  // namespace fftgb
