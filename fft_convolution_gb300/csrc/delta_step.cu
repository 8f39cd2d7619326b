// delta_step.cu -- the gated delta rule one token after the other, for
// decoding: a few tokens per sequence against a state that stays in HBM
// between calls.
//
// Per token  S <- e^g S;  u = beta (v - S^T k);  S <- S + k u^T;
//            o = scale S^T q.
// With S' the decayed state, S^T q = S'^T q + (k . q) u: both products with
// the state are taken in one walk over it, and one exchange between the
// threads gives every sum.  In a slow decay the state changes by k u +
// S (e^g - 1), added in one rounding: e^g itself would keep few digits of its
// distance from 1, an error that thousands of tokens add up; what rounding
// leaves out of u is carried along for the same reason.  In a quick one (g
// below kQuick, where less than half of S is left) it is k u + S e^g, each
// rounded at its own size: of S - S (1 - e^g) would only remain what the
// rounding of S leaves (g = -16: 20% of the state off).
//
// Reading and writing the fp32 state is nearly all the traffic (128 KB per
// head of 128 x 128, against under 1 KB for the token), so HBM bounds the
// kernel.  A block owns 32 columns of one head's state: their rows are whole
// 128-byte lines, a single sequence still spreads over dv / 32 blocks per
// head, and a block's share of the state fits the registers of 128 threads
// (4 columns and dk / 16 adjacent rows each), so the state is read once and
// written once however many tokens the call has.
#include "delta.cuh"

namespace fftgb {

constexpr int kStepThreads = 128, kStepCols = 32;
constexpr float kQuick = -0.6875f;  // -log 2, a little above

// N elements on a boundary of N elements (of 16 bytes, if that is less).
template <int N, typename T> __device__ __forceinline__ void load_whole(const T *p, float (&f)[N]) {
  constexpr int B = N * sizeof(T) < 16 ? N * sizeof(T) : 16, W = N * sizeof(T) / B;
  using Word = std::conditional_t<B == 16, uint4, uint2>;
  Word w[W];
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = reinterpret_cast<const Word *>(p)[i];
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = to_acc(reinterpret_cast<const T *>(w)[i]);
}

// Blocks per SM: what the registers of R rows allow.  (64 sequences with 16
// heads of 256 x 256: at 6 blocks, spilling 350 to 560 bytes, 113 us, at 3
// none, 90; of 192 x 192 78 and 67.  256 sequences with 32 heads of 96 x 96: 5
// blocks 143 us, 6 124, although a form or two spills 8 bytes.)
constexpr int step_blocks(int rows) { return rows > 8 ? 3 : 6; }

// VEC: the state goes by 16 bytes.  FULL: so do k, q and v, and all 16 R rows
// are there.  (One token of 128 sequences with 32 heads of 128 x 128: with
// elements of k and q loaded one by one 134 us, FULL 84: 95% of the copy rate;
// 5, 6 or 7 blocks per SM make 87, 84 and 84 us.)
template <typename T, int R, bool VEC, bool FULL>
__global__ void __launch_bounds__(kStepThreads, step_blocks(R))
delta_step_kernel(const DeltaArgs a) {
  __shared__ float4 red[2][4][8][3];
  const int tiles = (a.dv + kStepCols - 1) / kStepCols;
  const int tile = blockIdx.x % tiles;
  const long long bh = blockIdx.x / tiles;
  const int h = (int)(bh % a.vheads);
  const long long b = bh / a.vheads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cg = lane & 7;                       // 4 columns
  const int rg = warp * 4 + (lane >> 3);         // R rows
  const int r0 = rg * R, rows = FULL ? R : a.dk - r0;  // (there may be fewer, or none)
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

  float2 s[R][2];
  const long long s0 = (long long)r0 * a.dv + c0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (sin && i < rows) {
      const float *p = sin + s0 + (long long)i * a.dv;
      if constexpr (VEC) {
        if (c0 < a.dv) f = *reinterpret_cast<const float4 *>(p);
      } else {
        if (c0 < a.dv) f.x = p[0];
        if (c0 + 1 < a.dv) f.y = p[1];
        if (c0 + 2 < a.dv) f.z = p[2];
        if (c0 + 3 < a.dv) f.w = p[3];
      }
    }
    s[i][0] = make_float2(f.x, f.y);
    s[i][1] = make_float2(f.z, f.w);
  }

  const T *q = static_cast<const T *>(a.q) + b * a.sq.seq + hk * a.sq.head;
  const T *k = static_cast<const T *>(a.k) + b * a.sk.seq + hk * a.sk.head;
  const T *v = static_cast<const T *>(a.v) + b * a.sv.seq + h * a.sv.head;
  const float *g = a.g + b * a.sg.seq + h * a.sg.head;
  const float *beta = a.beta + b * a.sb.seq + h * a.sb.head;
  for (long long t = 0; t < a.tokens; ++t) {
    float kr[R], qr[R], vc[4];
    if constexpr (FULL) {
      load_whole(k + t * a.sk.tok + r0, kr);
      load_whole(q + t * a.sq.tok + r0, qr);
      vc[0] = vc[1] = vc[2] = vc[3] = 0.0f;
      if (c0 < a.dv) load_whole(v + t * a.sv.tok + c0, vc);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        kr[i] = i < rows ? to_acc(k[t * a.sk.tok + r0 + i]) : 0.0f;
        qr[i] = i < rows ? to_acc(q[t * a.sq.tok + r0 + i]) : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) vc[j] = c0 + j < a.dv ? to_acc(v[t * a.sv.tok + c0 + j]) : 0.0f;
    }
    const float gt = g[t * a.sg.tok], bt = beta[t * a.sb.tok];
    // S e^g = S decay + S whole.  Where k and q come element by element: after
    // the barrier, when fewer registers are live, and without a branch on g (256
    // sequences with 32 heads of 96 x 96: 124 us in bf16, 112 in fp32; before it
    // 132 and 112, with a branch 133 and 130).  Else here, with the branch, as
    // the state is still on its way (one token of 128 sequences: 84 us; without
    // the branch 85.5, after the barrier 86).
    const bool slow = gt > kQuick;
    float decay, whole;
    auto forget = [&]() {
      const float less = expm1f(gt), left = expf(gt);
      decay = slow ? less : left;
      whole = slow ? 1.0f : 0.0f;
    };
    if constexpr (FULL) {
      decay = slow ? expm1f(gt) : expf(gt);
      whole = slow ? 1.0f : 0.0f;
    }
    // S^T k and S^T q of the 4 columns (S before its decay), k . q
    float2 sk[2], sq[2];
    sk[0] = sk[1] = sq[0] = sq[1] = make_float2(0.0f, 0.0f);
    float kq = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sk[j] = fma2(both(kr[i]), s[i][j], sk[j]);
        sq[j] = fma2(both(qr[i]), s[i][j], sq[j]);
      }
      kq = fmaf(kr[i], qr[i], kq);
    }
    float sum[12] = {sk[0].x, sk[0].y, sk[1].x, sk[1].y, sq[0].x, sq[0].y, sq[1].x, sq[1].y, kq};
#pragma unroll
    for (int j = 0; j < 9; ++j) {
      sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 8);
      sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 16);
    }
    float4(*rd)[8][3] = red[t & 1];
    if (lane < 8)
#pragma unroll
      for (int j = 0; j < 3; ++j)
        rd[warp][cg][j] = make_float4(sum[4 * j], sum[4 * j + 1], sum[4 * j + 2], sum[4 * j + 3]);
    __syncthreads();  // the two halves of `red` alternate: one barrier per token
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const float4 w0 = rd[0][cg][j], w1 = rd[1][cg][j], w2 = rd[2][cg][j], w3 = rd[3][cg][j];
      sum[4 * j] = (w0.x + w1.x) + (w2.x + w3.x);
      sum[4 * j + 1] = (w0.y + w1.y) + (w2.y + w3.y);
      sum[4 * j + 2] = (w0.z + w1.z) + (w2.z + w3.z);
      sum[4 * j + 3] = (w0.w + w1.w) + (w2.w + w3.w);
    }
    if constexpr (!FULL) forget();
    float u[4], ur[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // u = beta (v - S'^T k) and what its rounding leaves out
      const float held = fmaf(decay, sum[j], whole * sum[j]), miss = vc[j] - held;
      const float back = miss - vc[j];
      const float rest = (vc[j] - (miss - back)) - (held + back);
      u[j] = bt * miss;
      ur[j] = fmaf(bt, miss, -u[j]) + bt * rest;
      if (rg == 0 && c0 + j < a.dv)
        o[t * ostep + c0 + j] =
            from_acc<T>(a.scale * fmaf(sum[8], u[j], fmaf(decay, sum[4 + j], whole * sum[4 + j])));
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 ku = make_float2(u[2 * j], u[2 * j + 1]), kur = make_float2(ur[2 * j], ur[2 * j + 1]);
        const float2 change =
            fma2(both(kr[i]), ku, fma2(both(kr[i]), kur, mul2(both(decay), s[i][j])));
        s[i][j] = fma2(s[i][j], both(whole), change);
      }
  }

  if (!sout) return;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i >= rows) continue;
    float *p = sout + s0 + (long long)i * a.dv;
    if constexpr (VEC) {
      if (c0 < a.dv)
        *reinterpret_cast<float4 *>(p) = make_float4(s[i][0].x, s[i][0].y, s[i][1].x, s[i][1].y);
    } else {
      if (c0 < a.dv) p[0] = s[i][0].x;
      if (c0 + 1 < a.dv) p[1] = s[i][0].y;
      if (c0 + 2 < a.dv) p[2] = s[i][1].x;
      if (c0 + 3 < a.dv) p[3] = s[i][1].y;
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
  // rows of k, q and v on 16-byte boundaries
  const bool whole = vec && vec_rows<T>(a.k, a.sk) && vec_rows<T>(a.q, a.sq) && vec_rows<T>(a.v, a.sv);
  auto pick = [&](auto rows) {
    constexpr int R = decltype(rows)::value;
    if (whole && a.dk == 16 * R) return run(delta_step_kernel<T, R, true, true>);
    return vec ? run(delta_step_kernel<T, R, true, false>) : run(delta_step_kernel<T, R, false, false>);
  };
  if (a.dk <= 64) return pick(std::integral_constant<int, 4>());
  if (a.dk <= 128) return pick(std::integral_constant<int, 8>());
  return pick(std::integral_constant<int, 16>());
}

cudaError_t launch_delta_step(int dtype, const DeltaArgs &a, cudaStream_t st) {
  if (dtype == FFT_ELEM_F32) return delta_step_t<float>(a, st);
  if (dtype == FFT_ELEM_BF16) return delta_step_t<__nv_bfloat16>(a, st);
  return delta_step_t<__half>(a, st);
}

}  // namespace fftgb
