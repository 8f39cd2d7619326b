// seq_ops.cu -- the C ABI of the sequence-model operators: argument checks,
// workspace sizes and the calls of the kernel launchers.
#include <math.h>

#include "plan.h"
#include "seq.h"

using namespace fftgb;

namespace fftgb {

int sm_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int v = cache[dev].load(std::memory_order_acquire);
  if (v == 0 && cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
    cache[dev].store(v, std::memory_order_release);
  return v;
}

}  // namespace fftgb

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxElems = (int64_t)1 << 46;

bool elem_type(int dtype) { return dtype >= FFT_ELEM_F32 && dtype <= FFT_ELEM_F16; }

bool off_element(const void *p, int dtype) { return ((uintptr_t)p & (elem_bytes(dtype) - 1)) != 0; }

// The types and sizes of a layer normalisation.
int norm_check(int64_t rows, int64_t dim, int dtype, int wtype) {
  if (rows < 0 || dim <= 0 || !elem_type(dtype) || !elem_type(wtype)) return FFT_ERR_INVALID_ARG;
  if (wtype != dtype && (wtype != FFT_ELEM_F32 || dtype == FFT_ELEM_F64))
    return FFT_ERR_UNSUPPORTED;
  if (dim > kMaxDim || rows > kMaxElems / dim) return FFT_ERR_UNSUPPORTED;
  return FFT_OK;
}

int finish(cudaError_t e) { return e == cudaSuccess ? FFT_OK : cuda_fail(e); }

int clip_check(int64_t count, const void *const *in, const int64_t *numel, const int *dtype) {
  if (count < 0 || (count > 0 && (!in || !numel || !dtype))) return FFT_ERR_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i) {
    if (numel[i] < 0 || !elem_type(dtype[i]) || (numel[i] > 0 && !in[i]))
      return FFT_ERR_INVALID_ARG;
    if (numel[i] > kMaxElems) return FFT_ERR_UNSUPPORTED;
    if (off_element(in[i], dtype[i])) return FFT_ERR_MISALIGNED;
  }
  return FFT_OK;
}

DeltaStride stride(const int64_t s[3]) { return DeltaStride{s[0], s[1], s[2]}; }

constexpr int64_t kDeltaMaxDk = 128;

// Sizes and types of a call of the delta rule.
int delta_sizes(const fft_delta_desc *d, int64_t max_dk, DeltaArgs *a) {
  if (!d) return FFT_ERR_INVALID_ARG;
  if (d->batch < 0 || d->tokens < 0 || d->kheads <= 0 || d->vheads <= 0 || d->dk <= 0 ||
      d->dv <= 0 || d->vheads % d->kheads != 0 || !elem_type(d->dtype) || !isfinite(d->scale))
    return FFT_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (d->q_stride[i] < 0 || d->k_stride[i] < 0 || d->v_stride[i] < 0 || d->g_stride[i] < 0 ||
        d->beta_stride[i] < 0)
      return FFT_ERR_INVALID_ARG;
  if (d->dtype == FFT_ELEM_F64 || d->dk > max_dk || d->dv > 65536 || d->vheads > 65536 ||
      d->tokens > 0x7fffffff || d->batch > ((int64_t)1 << 24) ||
      d->batch > 0x7fffffff / (d->vheads * ((d->dv + 31) / 32)) ||
      (d->tokens > 0 && d->batch > kMaxElems / (d->tokens * d->vheads)))
    return FFT_ERR_UNSUPPORTED;
  *a = DeltaArgs{};
  a->sq = stride(d->q_stride);
  a->sk = stride(d->k_stride);
  a->sv = stride(d->v_stride);
  a->sg = stride(d->g_stride);
  a->sb = stride(d->beta_stride);
  a->batch = d->batch;
  a->tokens = d->tokens;
  a->kheads = (int)d->kheads;
  a->vheads = (int)d->vheads;
  a->dk = (int)d->dk;
  a->dv = (int)d->dv;
  a->terms = d->dtype == FFT_ELEM_F32 ? 2 : 1;
  a->scale = (float)d->scale;
  a->clear = d->clear_rows != 0;
  return FFT_OK;
}

// Those and the inputs.
int delta_check(const fft_delta_desc *d, int64_t max_dk, const void *q, const void *k,
                const void *v, const float *g, const float *beta, DeltaArgs *a) {
  const int rc = delta_sizes(d, max_dk, a);
  if (rc != FFT_OK) return rc;
  if (d->batch > 0 && d->tokens > 0 && (!q || !k || !v || !g || !beta))
    return FFT_ERR_INVALID_ARG;
  if (off_element(q, d->dtype) || off_element(k, d->dtype) || off_element(v, d->dtype) ||
      off_element(g, FFT_ELEM_F32) || off_element(beta, FFT_ELEM_F32))
    return FFT_ERR_MISALIGNED;
  a->q = q;
  a->k = k;
  a->v = v;
  a->g = g;
  a->beta = beta;
  return FFT_OK;
}

// Grids of the kernels over all chunks, and of the gradients' two scans.
int delta_chunks_check(const DeltaArgs &a, bool packed) {
  const int64_t chunks = packed ? (a.tokens + 63 * a.batch) / 64 : a.batch * ((a.tokens + 63) / 64);
  return chunks > 0x3fffffff / a.vheads ? FFT_ERR_UNSUPPORTED : FFT_OK;
}

}  // namespace

extern "C" {

int fft_layer_norm(const void *x, int64_t ldx, const void *w, const void *b, void *y, int64_t ldy,
                   void *mean, void *rstd, int64_t rows, int64_t dim, double eps, int dtype,
                   int wtype, void *stream) {
  const int rc = norm_check(rows, dim, dtype, wtype);
  if (rc != FFT_OK) return rc;
  if (!(eps >= 0.0)) return FFT_ERR_INVALID_ARG;
  if (rows == 0) return FFT_OK;
  if (!x || !y || ldx < dim || ldy < dim || (x == y && ldx != ldy)) return FFT_ERR_INVALID_ARG;
  const int stype = dtype == FFT_ELEM_F64 ? FFT_ELEM_F64 : FFT_ELEM_F32;
  if (off_element(x, dtype) || off_element(y, dtype) || off_element(w, wtype) ||
      off_element(b, wtype) || off_element(mean, stype) || off_element(rstd, stype))
    return FFT_ERR_MISALIGNED;
  const LayerNormArgs a{x, w, b, y, mean, rstd, rows, ldx, ldy, (int)dim, eps, wtype};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case FFT_ELEM_F32: return finish(launch_layer_norm<float>(a, st));
    case FFT_ELEM_F64: return finish(launch_layer_norm<double>(a, st));
    case FFT_ELEM_BF16: return finish(launch_layer_norm<__nv_bfloat16>(a, st));
    default: return finish(launch_layer_norm<__half>(a, st));
  }
}

size_t fft_layer_norm_workspace_bytes(int64_t rows, int64_t dim, int dtype) {
  if (norm_check(rows, dim, dtype, dtype) != FFT_OK) return 0;
  return 2 * (size_t)layer_norm_partials(dtype, rows, (int)dim) * (size_t)dim *
         (dtype == FFT_ELEM_F64 ? 8 : 4);
}

int fft_layer_norm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                            const void *w, const void *mean, const void *rstd, void *dx,
                            int64_t lddx, void *dw, void *db, int64_t rows, int64_t dim,
                            int dtype, int wtype, void *workspace, size_t workspace_bytes,
                            void *stream) {
  const int rc = norm_check(rows, dim, dtype, wtype);
  if (rc != FFT_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (off_element(dw, wtype) || off_element(db, wtype)) return FFT_ERR_MISALIGNED;
  if (rows == 0) {  // empty sums
    const size_t bytes = (size_t)dim * elem_bytes(wtype);
    cudaError_t e = cudaSuccess;
    if (dw) e = cudaMemsetAsync(dw, 0, bytes, st);
    if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, bytes, st);
    return finish(e);
  }
  if (!dy || !x || !mean || !rstd || lddy < dim || ldx < dim || (dx && lddx < dim) ||
      (dx && dx == dy && lddx != lddy) || (dx && dx == x && lddx != ldx))
    return FFT_ERR_INVALID_ARG;
  const int stype = dtype == FFT_ELEM_F64 ? FFT_ELEM_F64 : FFT_ELEM_F32;
  if (off_element(dy, dtype) || off_element(x, dtype) || off_element(w, wtype) ||
      off_element(dx, dtype) || off_element(mean, stype) || off_element(rstd, stype))
    return FFT_ERR_MISALIGNED;
  if (!dx && !dw && !db) return FFT_OK;
  if (dw || db) {
    if (!workspace || workspace_bytes < fft_layer_norm_workspace_bytes(rows, dim, dtype))
      return FFT_ERR_INVALID_ARG;
    if (misaligned(workspace)) return FFT_ERR_MISALIGNED;
  }
  const LayerNormGradArgs a{dy, x,   w,    mean, rstd, dx, dw, db, rows, lddy, ldx, lddx, (int)dim,
                            wtype, (dw || db) ? workspace : nullptr};
  switch (dtype) {
    case FFT_ELEM_F32: return finish(launch_layer_norm_grad<float>(a, st));
    case FFT_ELEM_F64: return finish(launch_layer_norm_grad<double>(a, st));
    case FFT_ELEM_BF16: return finish(launch_layer_norm_grad<__nv_bfloat16>(a, st));
    default: return finish(launch_layer_norm_grad<__half>(a, st));
  }
}

size_t fft_grad_norm_workspace_bytes(int64_t count) {
  return count < 0 ? 0 : clip_workspace_bytes(count);
}

int fft_grad_norm(int64_t count, const void *const *in, const int64_t *numel, const int *dtype,
                  float *norm, void *workspace, size_t workspace_bytes, void *stream) {
  const int rc = clip_check(count, in, numel, dtype);
  if (rc != FFT_OK) return rc;
  if (!norm || !workspace || workspace_bytes < clip_workspace_bytes(count))
    return FFT_ERR_INVALID_ARG;
  if (misaligned(workspace) || off_element(norm, FFT_ELEM_F32)) return FFT_ERR_MISALIGNED;
  return finish(launch_clip(count, in, nullptr, numel, dtype, 0.0, 0.0, norm, workspace,
                            static_cast<cudaStream_t>(stream)));
}

int fft_clip_grad_norm(int64_t count, const void *const *in, void *const *out,
                       const int64_t *numel, const int *dtype, double max_norm, double eps,
                       float *norm, void *workspace, size_t workspace_bytes, void *stream) {
  const int rc = clip_check(count, in, numel, dtype);
  if (rc != FFT_OK) return rc;
  if ((count > 0 && !out) || !(max_norm >= 0.0) || !(eps >= 0.0) || !workspace ||
      workspace_bytes < clip_workspace_bytes(count))
    return FFT_ERR_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i) {
    if (numel[i] > 0 && !out[i]) return FFT_ERR_INVALID_ARG;
    if (off_element(out[i], dtype[i])) return FFT_ERR_MISALIGNED;
  }
  if (misaligned(workspace) || off_element(norm, FFT_ELEM_F32)) return FFT_ERR_MISALIGNED;
  void *const none[1] = {nullptr};
  return finish(launch_clip(count, in, count > 0 ? out : none, numel, dtype, max_norm, eps, norm,
                            workspace, static_cast<cudaStream_t>(stream)));
}

size_t fft_delta_rule_workspace_bytes(const fft_delta_desc *desc, int packed) {
  DeltaArgs a;
  if (delta_sizes(desc, kDeltaMaxDk, &a) != FFT_OK || delta_chunks_check(a, packed != 0) != FFT_OK)
    return 0;
  return delta_workspace_bytes(a, packed != 0);
}

int fft_delta_rule(const fft_delta_desc *desc, const void *q, const void *k, const void *v,
                   const float *g, const float *beta, const int32_t *offsets,
                   const float *initial_state, void *o, float *final_state, void *workspace,
                   size_t workspace_bytes, void *stream) {
  DeltaArgs a;
  int rc = delta_check(desc, kDeltaMaxDk, q, k, v, g, beta, &a);
  if (rc == FFT_OK) rc = delta_chunks_check(a, offsets != nullptr);
  if (rc != FFT_OK) return rc;
  a.clear = a.clear && offsets && a.tokens > 0;
  if (a.batch == 0 && !a.clear) return FFT_OK;
  if ((a.tokens > 0 && !o) ||
      (workspace_bytes < delta_workspace_bytes(a, offsets != nullptr)) ||
      (!workspace && delta_workspace_bytes(a, offsets != nullptr) > 0))
    return FFT_ERR_INVALID_ARG;
  if (misaligned(workspace) || off_element(o, desc->dtype) ||
      off_element(initial_state, FFT_ELEM_F32) || off_element(final_state, FFT_ELEM_F32) ||
      off_element(offsets, FFT_ELEM_F32))
    return FFT_ERR_MISALIGNED;
  a.offsets = offsets;
  a.state_in = initial_state;
  a.state_out = final_state;
  a.o = o;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.batch == 0)
    return finish(launch_delta_plan(offsets, 0, a.tokens, nullptr, nullptr,
                                    delta_clear(a, nullptr, elem_bytes(desc->dtype)), st));
  switch (desc->dtype) {
    case FFT_ELEM_F32: return finish(launch_delta<float>(a, workspace, st));
    case FFT_ELEM_BF16: return finish(launch_delta<__nv_bfloat16>(a, workspace, st));
    default: return finish(launch_delta<__half>(a, workspace, st));
  }
}

size_t fft_delta_rule_backward_workspace_bytes(const fft_delta_desc *desc, int packed) {
  DeltaArgs a;
  if (delta_sizes(desc, kDeltaMaxDk, &a) != FFT_OK || delta_chunks_check(a, packed != 0) != FFT_OK)
    return 0;
  return delta_grad_workspace_bytes(a, packed != 0);
}

int fft_delta_rule_backward(const fft_delta_desc *desc, const void *dout, const void *q,
                            const void *k, const void *v, const float *g, const float *beta,
                            const int32_t *offsets, const float *initial_state,
                            const float *dfinal_state, void *dq, void *dk, void *dv, float *dg,
                            float *dbeta, float *dinitial_state, void *workspace,
                            size_t workspace_bytes, void *stream) {
  DeltaArgs a;
  int rc = delta_check(desc, kDeltaMaxDk, q, k, v, g, beta, &a);
  if (rc == FFT_OK) rc = delta_chunks_check(a, offsets != nullptr);
  if (rc != FFT_OK) return rc;
  a.clear = a.clear && offsets && a.tokens > 0;
  if (a.batch == 0 && !a.clear) return FFT_OK;
  const size_t need = delta_grad_workspace_bytes(a, offsets != nullptr);
  if ((a.tokens > 0 && (!dout || !dq || !dk || !dv || !dg || !dbeta)) || workspace_bytes < need ||
      (!workspace && need > 0))
    return FFT_ERR_INVALID_ARG;
  for (const void *p : {dout, (const void *)dq, (const void *)dk, (const void *)dv})
    if (off_element(p, desc->dtype)) return FFT_ERR_MISALIGNED;
  for (const void *p : {(const void *)initial_state, (const void *)dfinal_state, (const void *)dg,
                        (const void *)dbeta, (const void *)dinitial_state, (const void *)offsets})
    if (off_element(p, FFT_ELEM_F32)) return FFT_ERR_MISALIGNED;
  if (misaligned(workspace)) return FFT_ERR_MISALIGNED;
  a.offsets = offsets;
  a.state_in = initial_state;
  const DeltaGradArgs ga{dout, dfinal_state, dq, dk, dv, dg, dbeta, dinitial_state};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.batch == 0)
    return finish(launch_delta_plan(offsets, 0, a.tokens, nullptr, nullptr,
                                    delta_clear(a, &ga, elem_bytes(desc->dtype)), st));
  switch (desc->dtype) {
    case FFT_ELEM_F32: return finish(launch_delta_grad<float>(a, ga, workspace, st));
    case FFT_ELEM_BF16: return finish(launch_delta_grad<__nv_bfloat16>(a, ga, workspace, st));
    default: return finish(launch_delta_grad<__half>(a, ga, workspace, st));
  }
}

int fft_delta_rule_step(const fft_delta_desc *desc, const void *q, const void *k, const void *v,
                        const float *g, const float *beta, float *state, const int32_t *slots,
                        int64_t pool, void *o, void *stream) {
  DeltaArgs a;
  const int rc = delta_check(desc, 256, q, k, v, g, beta, &a);
  if (rc != FFT_OK) return rc;
  if (pool < 0 || (!slots && pool < desc->batch)) return FFT_ERR_INVALID_ARG;
  if (desc->batch == 0 || desc->tokens == 0) return FFT_OK;
  if (!o || (pool > 0 && !state)) return FFT_ERR_INVALID_ARG;
  if (off_element(o, desc->dtype) || off_element(state, FFT_ELEM_F32) ||
      off_element(slots, FFT_ELEM_F32))
    return FFT_ERR_MISALIGNED;
  a.state_in = state;
  a.state_out = state;
  a.slots = slots;
  a.pool = pool;
  a.o = o;
  return finish(launch_delta_step(desc->dtype, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
