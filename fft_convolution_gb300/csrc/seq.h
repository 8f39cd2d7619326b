// seq.h -- declarations shared by the sequence-model operators (layer
// normalisation, gradient clipping, the gated delta rule): element types,
// conversions, and the kernel launchers behind the C ABI of seq_ops.cu.
// Not installed.
#pragma once

#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"

namespace fftgb {

inline size_t elem_bytes(int dtype) {
  return dtype == FFT_ELEM_F64 ? 8 : dtype == FFT_ELEM_F32 ? 4 : 2;
}

// Multiprocessors of the current device (0 if the query fails).
int sm_count();

// ---- layer normalisation (layer_norm_*.cu) -----------------------------------

struct LayerNormArgs {
  const void *x, *w, *b;  // w, b may be null (1 and 0)
  void *y;
  void *mean, *rstd;  // fp32 (fp64 rows: fp64); may be null
  long long rows, ldx, ldy;
  int dim;
  double eps;
  int wtype;
};
struct LayerNormGradArgs {
  const void *dy, *x, *w, *mean, *rstd;  // w may be null
  void *dx, *dw, *db;                    // each may be null
  long long rows, lddy, ldx, lddx;
  int dim;
  int wtype;
  void *partial;  // 2 x layer_norm_partials() x dim accumulators
};
// Rows of partial sums of the weight's gradient that the backward pass leaves.
int layer_norm_partials(int dtype, long long rows, int dim);
template <typename T> cudaError_t launch_layer_norm(const LayerNormArgs &a, cudaStream_t st);
template <typename T> cudaError_t launch_layer_norm_grad(const LayerNormGradArgs &a,
                                                         cudaStream_t st);

// ---- gradient clipping (clip.cu) ---------------------------------------------

size_t clip_workspace_bytes(long long count);
cudaError_t launch_clip(long long count, const void *const *in, void *const *out,
                        const int64_t *numel, const int *dtype, double max_norm, double eps,
                        float *norm, void *workspace, cudaStream_t st);

// ---- the gated delta rule (delta_*.cu) ------------------------------------------

// Strides in elements: sequence (unused for packed rows), token, head.
struct DeltaStride {
  long long seq, tok, head;
};
struct DeltaArgs {
  const void *q, *k, *v;
  const float *g, *beta;
  DeltaStride sq, sk, sv, sg, sb;
  const int *offsets;     // packed rows: batch + 1 first rows; else null
  const float *state_in;  // may be null (zero)
  float *state_out;       // may be null
  void *o;                // contiguous [sequence][token][head][dv]
  long long batch, tokens;
  int kheads, vheads, dk, dv;
  int terms;  // fp16 values that hold one element of q and k (2: fp32)
  float scale;
  bool clear;  // packed rows that belong to no sequence: results of 0
  // Single tokens: the sequence's row of a pool of `pool` states (null: row = sequence).
  const int *slots;
  long long pool;
};
// The gradients' own arrays: contiguous, laid out like the inputs without
// strides ([sequence][token][head][..], packed: [row][head][..]).
struct DeltaGradArgs {
  const void *dout;
  const float *dfinal;  // may be null (zero)
  void *dq, *dk, *dv;
  float *dg, *dbeta, *dinitial;  // dinitial may be null
};
cudaError_t launch_delta_step(int dtype, const DeltaArgs &a, cudaStream_t st);
// Whole sequences, in chunks; `workspace` holds delta_workspace_bytes().
size_t delta_workspace_bytes(const DeltaArgs &a, bool packed);
template <typename T>
cudaError_t launch_delta(const DeltaArgs &a, void *workspace, cudaStream_t st);
size_t delta_grad_workspace_bytes(const DeltaArgs &a, bool packed);
template <typename T>
cudaError_t launch_delta_grad(const DeltaArgs &a, const DeltaGradArgs &g, void *workspace,
                              cudaStream_t st);
// Packed arrays whose rows of no sequence are to be 0.
struct DeltaClear {
  void *p[5];
  long long row_bytes[5];
  int count;
};
// The results of a call (g: of the gradients); none unless a.clear.
DeltaClear delta_clear(const DeltaArgs &a, const DeltaGradArgs *g, size_t elem);
// Fills row0 and chunk0 (batch + 1 entries each; null: not wanted) from offsets
// and clears rows (delta_plan.cu).
cudaError_t launch_delta_plan(const int *offsets, long long batch, long long tokens, int *row0,
                              int *chunk0, const DeltaClear &clear, cudaStream_t st);

// ---- embedding of tokens (embed.cu) ----------------------------------------------

struct EmbedArgs {
  const void *ids;
  int id_bytes;  // 4 or 8
  const void *table;
  void *y;
  long long tokens, rows, ldt, ldy;
  int dim;
  double scale;
};
struct EmbedGradArgs {
  const void *dy, *ids;
  int id_bytes;
  void *dtable;  // rows x dim
  long long tokens, rows, lddy;
  int dim;
  double scale;
  bool add;  // to what dtable holds
};
// The tokens sorted by row, and bytes to clear meanwhile.
struct EmbedSortArgs {
  const void *ids;
  int id_bytes;
  long long tokens, rows;
  int passes, bits;
  unsigned *key[2], *pos[2];  // row (tokens of no row: `rows`) and token; pass p reads [p & 1]
  void *fill;
  long long fill_bytes;
  unsigned *crossing;  // set to 0
  unsigned blocks;     // of a cluster
};
struct EmbedSumArgs {
  const void *dy;
  const unsigned *key, *pos;
  unsigned *crossing, *list;  // how many runs go on behind their first piece, and those pieces
  void *dtable, *partial;     // partial: [piece][head, tail][ldp] accumulators
  long long tokens, rows, lddy, ldp;
  int dim;
  int piece;  // tokens of a piece
  double scale;
  bool add;
};
size_t embed_workspace_bytes(long long tokens, int dim, int dtype);
cudaError_t launch_embed(int dtype, const EmbedArgs &a, cudaStream_t st);
cudaError_t launch_embed_grad(int dtype, int ttype, const EmbedGradArgs &a, void *workspace,
                              cudaStream_t st);

// ---- the gated linear recurrence (recur_*.cu) ---------------------------------------

// How long waits inside kernels may take, in clocks, and (FFT_OPT_STARVED_WAIT) which barrier
// of the first block never completes: 0, none.
struct Waits {
  long long limit;
  int starved;
};
inline Waits waits_now() {
  const long long starved = option(FFT_OPT_STARVED_WAIT);
  return starved > 0 ? Waits{1ll << 21, (int)starved} : Waits{8000000000ll, 0};  // about 4 s
}

// Strides in elements: sequence (unused for packed rows) and token.
struct RecurStride {
  long long seq, tok;
};
struct RecurArgs {
  const void *x, *g, *beta;  // beta may be null (1)
  RecurStride sx, sg, sb;
  const int *offsets;      // packed rows: batch + 1 first rows; else null
  const float *state_in;   // may be null (zero)
  float *state_out;        // may be null
  void *y;                 // contiguous [sequence][token][channel]; the gradient reads it
  long long batch, tokens;
  int channels;
  bool clear;  // packed rows of no sequence: results of 0
  int blocks;  // of a cluster, which share a sequence's tokens
  int *rows;   // packed, many sequences: 2 (batch + 1) entries, the first half of which
               // become the sequences' first rows; else null
  Waits waits;
  // Single tokens: the sequence's row of a pool of `pool` states (null: row = sequence).
  const int *slots;
  long long pool;
  // The gradients' own arrays, contiguous like y.
  const void *dy;
  const float *dfinal;  // may be null (zero)
  void *dx, *dg, *dbeta;
  float *dinitial;  // may be null
};
size_t recur_workspace_bytes(long long batch, bool packed);
// g and beta of type float where gfloat, else of type T.
template <typename T> cudaError_t launch_recur(const RecurArgs &a, bool gfloat, cudaStream_t st);
template <typename T>
cudaError_t launch_recur_grad(const RecurArgs &a, bool gfloat, cudaStream_t st);
template <typename T>
cudaError_t launch_recur_step(const RecurArgs &a, bool gfloat, cudaStream_t st);

// ---- cross entropy of a linear layer (xent.cu) --------------------------------------

struct XentArgs {
  const void *x, *w;  // tokens x dim, vocabulary x dim
  long long ldx, ldw;
  const void *targets;
  int target_bytes;  // 4 or 8
  long long tokens, vocabulary;
  int dim;
  float *loss, *lse;  // the gradients read lse
  // The gradients' own arrays.
  const float *dloss;
  void *dx, *dw;  // contiguous; each may be null
};
size_t xent_workspace_bytes(int dtype, const XentArgs &a, bool grad);
cudaError_t launch_xent(int dtype, const XentArgs &a, void *workspace, cudaStream_t st);
cudaError_t launch_xent_grad(int dtype, const XentArgs &a, void *workspace, cudaStream_t st);

// ---- chains of kernels -----------------------------------------------------------

// Launches a kernel of a call.  With `chained` it follows another kernel of the
// same call, and its blocks may start before that one has finished (programmatic
// dependent launch): such kernels begin with after_previous(), and the one before
// lets them start with let_next().  `cluster` blocks form a cluster (1: none).
template <typename... P, typename... A>
cudaError_t launch_kernel(bool chained, void (*kern)(P...), unsigned grid, dim3 block, size_t smem,
                          unsigned cluster, cudaStream_t st, const A &...args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (chained) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = cluster;
    at[n].val.clusterDim.y = 1;
    at[n++].val.clusterDim.z = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}
#ifdef __CUDACC__
// Every kernel before this one in the call has finished, its writes are seen.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// The next kernel's blocks may start once all of this one's have come here.
__device__ __forceinline__ void let_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
#endif

// ---- element conversions -----------------------------------------------------

#ifdef __CUDACC__
__device__ __forceinline__ float to_acc(float v) { return v; }
__device__ __forceinline__ double to_acc(double v) { return v; }
__device__ __forceinline__ float to_acc(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_acc(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_acc(float v);
template <> __device__ __forceinline__ float from_acc<float>(float v) { return v; }
template <> __device__ __forceinline__ double from_acc<double>(float v) { return (double)v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_acc<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ __half from_acc<__half>(float v) {
  return __float2half_rn(v);
}
template <typename T> __device__ __forceinline__ T from_acc(double v);
template <> __device__ __forceinline__ double from_acc<double>(double v) { return v; }
template <> __device__ __forceinline__ float from_acc<float>(double v) { return (float)v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_acc<__nv_bfloat16>(double v) {
  return __double2bfloat16(v);
}
template <> __device__ __forceinline__ __half from_acc<__half>(double v) {
  return __double2half(v);
}

// Accumulator type of an element type.
template <typename T> struct Acc { using type = float; };
template <> struct Acc<double> { using type = double; };

// Element i of an array whose type is known at run time only (the branch is
// the same for every thread).
__device__ __forceinline__ float load_any(const void *p, int dtype, long long i) {
  if (dtype == FFT_ELEM_F32) return static_cast<const float *>(p)[i];
  if (dtype == FFT_ELEM_BF16) return to_acc(static_cast<const __nv_bfloat16 *>(p)[i]);
  if (dtype == FFT_ELEM_F16) return to_acc(static_cast<const __half *>(p)[i]);
  return (float)static_cast<const double *>(p)[i];
}
template <typename A>
__device__ __forceinline__ void store_any(void *p, int dtype, long long i, A v) {
  if (dtype == FFT_ELEM_F32) static_cast<float *>(p)[i] = from_acc<float>(v);
  else if (dtype == FFT_ELEM_BF16) static_cast<__nv_bfloat16 *>(p)[i] = from_acc<__nv_bfloat16>(v);
  else if (dtype == FFT_ELEM_F16) static_cast<__half *>(p)[i] = from_acc<__half>(v);
  else static_cast<double *>(p)[i] = from_acc<double>(v);
}

// 16 bytes of elements.
template <typename T> struct alignas(16) Vec16 {
  static constexpr int N = 16 / sizeof(T);
  T v[N];
};
// The elements of 16 bytes, and back.
template <typename T> __device__ __forceinline__ void unpack(uint4 w, float (&f)[4]) {
  f[0] = __uint_as_float(w.x);
  f[1] = __uint_as_float(w.y);
  f[2] = __uint_as_float(w.z);
  f[3] = __uint_as_float(w.w);
}
template <typename T> __device__ __forceinline__ void unpack(uint4 w, float (&f)[8]) {
  const unsigned r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 x;
    if constexpr (std::is_same<T, __half>::value) {
      x = __half22float2(*reinterpret_cast<const __half2 *>(&r[i]));
    } else {
      x.x = __uint_as_float(r[i] << 16);
      x.y = __uint_as_float(r[i] & 0xffff0000u);
    }
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}
template <typename T> __device__ __forceinline__ void unpack(uint4 w, double (&f)[2]) {
  f[0] = __hiloint2double((int)w.y, (int)w.x);
  f[1] = __hiloint2double((int)w.w, (int)w.z);
}
template <typename T> __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}
template <typename T> __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  unsigned r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, __half>::value) {
      const __half2 x = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      r[i] = *reinterpret_cast<const unsigned *>(&x);
    } else {
      const __nv_bfloat162 x = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      r[i] = *reinterpret_cast<const unsigned *>(&x);
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
template <typename T> __device__ __forceinline__ uint4 pack(const double (&f)[2]) {
  return make_uint4((unsigned)__double2loint(f[0]), (unsigned)__double2hiint(f[0]),
                    (unsigned)__double2loint(f[1]), (unsigned)__double2hiint(f[1]));
}
#endif

}  // namespace fftgb
