// model_ops.cu -- the C ABI of the embedding, the gated linear recurrence and
// the cross entropy of a linear layer: argument checks, workspace sizes and the
// calls of the kernel launchers.
#include <math.h>

#include "plan.h"
#include "seq.h"

using namespace fftgb;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 30;
constexpr int64_t kMaxElems = (int64_t)1 << 46;
constexpr int64_t kMaxInt = 0x7fffffff;

bool elem_type(int dtype) { return dtype >= FFT_ELEM_F32 && dtype <= FFT_ELEM_F16; }
bool off_element(const void *p, int dtype) { return ((uintptr_t)p & (elem_bytes(dtype) - 1)) != 0; }
bool off_bytes(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) != 0; }
int finish(cudaError_t e) { return e == cudaSuccess ? FFT_OK : cuda_fail(e); }

int embed_sizes(int64_t tokens, int64_t rows, int64_t dim, int dtype) {
  if (tokens < 0 || rows <= 0 || dim <= 0 || !elem_type(dtype)) return FFT_ERR_INVALID_ARG;
  if (tokens > kMaxInt - 63 || rows > kMaxInt || dim > kMaxDim || rows > kMaxElems / dim ||
      tokens > kMaxElems / dim)
    return FFT_ERR_UNSUPPORTED;
  return FFT_OK;
}

RecurStride stride(const int64_t s[2]) { return RecurStride{s[0], s[1]}; }

// Sizes and types of a call of the recurrence. Packed: `tokens` are those of all sequences.
int recur_sizes(const fft_recurrence_desc *d, bool packed, RecurArgs *a) {
  if (!d || d->batch < 0 || d->tokens < 0 || d->channels <= 0 || !elem_type(d->dtype) ||
      !elem_type(d->gtype))
    return FFT_ERR_INVALID_ARG;
  for (int i = 0; i < 2; ++i)
    if (d->x_stride[i] < 0 || d->g_stride[i] < 0 || d->beta_stride[i] < 0)
      return FFT_ERR_INVALID_ARG;
  if (d->dtype == FFT_ELEM_F64 || (d->gtype != d->dtype && d->gtype != FFT_ELEM_F32) ||
      d->tokens > kMaxInt || d->channels > kMaxDim || d->batch > ((int64_t)1 << 24) ||
      (d->batch > 0 && (d->channels + 127) / 128 > kMaxInt / 8 / d->batch) ||
      (d->tokens > 0 && (packed ? 1 : d->batch) > kMaxElems / d->tokens / d->channels))
    return FFT_ERR_UNSUPPORTED;
  *a = RecurArgs{};
  a->sx = stride(d->x_stride);
  a->sg = stride(d->g_stride);
  a->sb = stride(d->beta_stride);
  a->batch = d->batch;
  a->tokens = d->tokens;
  a->channels = (int)d->channels;
  a->clear = d->clear_rows != 0;
  return FFT_OK;
}

// Those and the inputs.
int recur_check(const fft_recurrence_desc *d, const void *x, const void *g, const void *beta,
                bool x_used, bool packed, RecurArgs *a) {
  const int rc = recur_sizes(d, packed, a);
  if (rc != FFT_OK) return rc;
  if (d->batch > 0 && d->tokens > 0 && ((x_used && !x) || !g)) return FFT_ERR_INVALID_ARG;
  if (off_element(x, d->dtype) || off_element(g, d->gtype) || off_element(beta, d->gtype))
    return FFT_ERR_MISALIGNED;
  a->x = x;
  a->g = g;
  a->beta = beta;
  return FFT_OK;
}

// Where the first rows of many packed sequences are put.
int recur_workspace(RecurArgs *a, void *workspace, size_t workspace_bytes) {
  const size_t need = a->batch > 0 ? recur_workspace_bytes(a->batch, a->offsets != nullptr) : 0;
  if (need == 0) return FFT_OK;
  if (!workspace || workspace_bytes < need) return FFT_ERR_INVALID_ARG;
  if (misaligned(workspace)) return FFT_ERR_MISALIGNED;
  a->rows = static_cast<int *>(workspace);
  return FFT_OK;
}

// Packed rows without a sequence: zeros everywhere.
cudaError_t clear_all(const RecurArgs &a, void *p, int dtype, cudaStream_t st) {
  if (!p) return cudaSuccess;
  return cudaMemsetAsync(p, 0, (size_t)a.tokens * a.channels * elem_bytes(dtype), st);
}

int xent_check(const void *x, int64_t ldx, const void *w, int64_t ldw, int64_t tokens,
               int64_t vocabulary, int64_t dim, int dtype, XentArgs *a) {
  if (tokens < 0 || vocabulary <= 0 || dim <= 0 || !elem_type(dtype)) return FFT_ERR_INVALID_ARG;
  if (dtype == FFT_ELEM_F64 || tokens > ((int64_t)1 << 24) || vocabulary > ((int64_t)1 << 24) ||
      dim > ((int64_t)1 << 20) || ldx > ((int64_t)1 << 31) || ldw > ((int64_t)1 << 31) ||
      ((tokens + 255) / 256) * ((vocabulary + 255) / 256) > kMaxInt ||
      ((tokens + vocabulary + 511) / 256) * ((dim + 255) / 256) > kMaxInt / 32)
    return FFT_ERR_UNSUPPORTED;
  if (ldx < dim || ldw < dim) return FFT_ERR_INVALID_ARG;
  *a = XentArgs{};
  a->x = x;
  a->w = w;
  a->ldx = ldx;
  a->ldw = ldw;
  a->tokens = tokens;
  a->vocabulary = vocabulary;
  a->dim = (int)dim;
  return FFT_OK;
}

}  // namespace

extern "C" {

int fft_embedding(const void *ids, int id_bytes, const void *table, int64_t ldt, void *y,
                  int64_t ldy, int64_t tokens, int64_t rows, int64_t dim, double scale, int dtype,
                  void *stream) {
  const int rc = embed_sizes(tokens, rows, dim, dtype);
  if (rc != FFT_OK) return rc;
  if ((id_bytes != 4 && id_bytes != 8) || !isfinite(scale)) return FFT_ERR_INVALID_ARG;
  if (tokens == 0) return FFT_OK;
  if (!ids || !table || !y || ldt < dim || ldy < dim) return FFT_ERR_INVALID_ARG;
  if (ldt > kMaxElems / rows || ldy > kMaxElems / tokens) return FFT_ERR_UNSUPPORTED;
  if (off_bytes(ids, id_bytes) || off_element(table, dtype) || off_element(y, dtype))
    return FFT_ERR_MISALIGNED;
  const EmbedArgs a{ids, id_bytes, table, y, tokens, rows, ldt, ldy, (int)dim, scale};
  return finish(launch_embed(dtype, a, static_cast<cudaStream_t>(stream)));
}

size_t fft_embedding_workspace_bytes(int64_t tokens, int64_t dim, int dtype) {
  return embed_sizes(tokens, 1, dim, dtype) == FFT_OK
             ? embed_workspace_bytes(tokens, (int)dim, dtype)
             : 0;
}

int fft_embedding_backward(const void *dy, int64_t lddy, const void *ids, int id_bytes,
                           void *dtable, int64_t tokens, int64_t rows, int64_t dim, double scale,
                           int add, int dtype, int ttype, void *workspace, size_t workspace_bytes,
                           void *stream) {
  const int rc = embed_sizes(tokens, rows, dim, dtype);
  if (rc != FFT_OK) return rc;
  if ((id_bytes != 4 && id_bytes != 8) || !isfinite(scale) || !elem_type(ttype) || !dtable)
    return FFT_ERR_INVALID_ARG;
  if (ttype != dtype && (ttype != FFT_ELEM_F32 || dtype == FFT_ELEM_F64))
    return FFT_ERR_UNSUPPORTED;
  // a block per four pieces of 16 tokens x 128 columns
  if ((tokens + 15) / 16 > 4 * kMaxInt / ((dim + 63) / 64)) return FFT_ERR_UNSUPPORTED;
  if (off_element(dtable, ttype)) return FFT_ERR_MISALIGNED;
  if (tokens > 0) {
    if (!dy || !ids || lddy < dim || !workspace ||
        workspace_bytes < embed_workspace_bytes(tokens, (int)dim, dtype))
      return FFT_ERR_INVALID_ARG;
    if (lddy > kMaxElems / tokens) return FFT_ERR_UNSUPPORTED;
    if (off_bytes(ids, id_bytes) || off_element(dy, dtype) || misaligned(workspace))
      return FFT_ERR_MISALIGNED;
  }
  const EmbedGradArgs a{dy, ids, id_bytes, dtable, tokens, rows, lddy, (int)dim, scale, add != 0};
  return finish(launch_embed_grad(dtype, ttype, a, workspace, static_cast<cudaStream_t>(stream)));
}

size_t fft_linear_recurrence_workspace_bytes(const fft_recurrence_desc *desc, int packed) {
  RecurArgs a;
  if (!desc || recur_sizes(desc, packed != 0, &a) != FFT_OK || a.batch == 0) return 0;
  return recur_workspace_bytes(a.batch, packed != 0);
}

int fft_linear_recurrence(const fft_recurrence_desc *desc, const void *x, const void *g,
                          const void *beta, const int32_t *offsets, const float *initial_state,
                          void *y, float *final_state, void *workspace, size_t workspace_bytes,
                          void *stream) {
  RecurArgs a;
  int rc = recur_check(desc, x, g, beta, true, offsets != nullptr, &a);
  if (rc != FFT_OK) return rc;
  a.clear = a.clear && offsets && a.tokens > 0;
  if (a.batch == 0 && !a.clear) return FFT_OK;
  if (a.tokens > 0 && !y) return FFT_ERR_INVALID_ARG;
  if (off_element(y, desc->dtype) || off_element(initial_state, FFT_ELEM_F32) ||
      off_element(final_state, FFT_ELEM_F32) || off_element(offsets, FFT_ELEM_F32))
    return FFT_ERR_MISALIGNED;
  a.offsets = offsets;
  a.state_in = initial_state;
  a.state_out = final_state;
  a.y = y;
  rc = recur_workspace(&a, workspace, workspace_bytes);
  if (rc != FFT_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.batch == 0) return finish(clear_all(a, y, desc->dtype, st));
  const bool gf = desc->gtype == FFT_ELEM_F32;
  switch (desc->dtype) {
    case FFT_ELEM_F32: return finish(launch_recur<float>(a, gf, st));
    case FFT_ELEM_BF16: return finish(launch_recur<__nv_bfloat16>(a, gf, st));
    default: return finish(launch_recur<__half>(a, gf, st));
  }
}

int fft_linear_recurrence_backward(const fft_recurrence_desc *desc, const void *dy, const void *x,
                                   const void *g, const void *beta, const void *y,
                                   const int32_t *offsets, const float *initial_state,
                                   const float *dfinal_state, void *dx, void *dg, void *dbeta,
                                   float *dinitial_state, void *workspace,
                                   size_t workspace_bytes, void *stream) {
  RecurArgs a;
  int rc = recur_check(desc, x, g, beta, beta != nullptr, offsets != nullptr, &a);
  if (rc != FFT_OK) return rc;
  a.clear = a.clear && offsets && a.tokens > 0;
  if (a.batch == 0 && !a.clear) return FFT_OK;
  if (a.tokens > 0 && (!dy || !y || !dx || !dg || (beta && !dbeta))) return FFT_ERR_INVALID_ARG;
  for (const void *p : {dy, y, (const void *)dx})
    if (off_element(p, desc->dtype)) return FFT_ERR_MISALIGNED;
  for (const void *p : {(const void *)dg, (const void *)dbeta})
    if (off_element(p, desc->gtype)) return FFT_ERR_MISALIGNED;
  for (const void *p : {(const void *)initial_state, (const void *)dfinal_state,
                        (const void *)dinitial_state, (const void *)offsets})
    if (off_element(p, FFT_ELEM_F32)) return FFT_ERR_MISALIGNED;
  a.offsets = offsets;
  a.state_in = initial_state;
  a.y = const_cast<void *>(y);  // read only
  a.dy = dy;
  a.dfinal = dfinal_state;
  a.dx = dx;
  a.dg = dg;
  a.dbeta = beta ? dbeta : nullptr;
  a.dinitial = dinitial_state;
  rc = recur_workspace(&a, workspace, workspace_bytes);
  if (rc != FFT_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.batch == 0) {
    cudaError_t e = clear_all(a, dx, desc->dtype, st);
    if (e == cudaSuccess) e = clear_all(a, dg, desc->gtype, st);
    if (e == cudaSuccess) e = clear_all(a, a.dbeta, desc->gtype, st);
    return finish(e);
  }
  const bool gf = desc->gtype == FFT_ELEM_F32;
  switch (desc->dtype) {
    case FFT_ELEM_F32: return finish(launch_recur_grad<float>(a, gf, st));
    case FFT_ELEM_BF16: return finish(launch_recur_grad<__nv_bfloat16>(a, gf, st));
    default: return finish(launch_recur_grad<__half>(a, gf, st));
  }
}

int fft_linear_recurrence_step(const fft_recurrence_desc *desc, const void *x, const void *g,
                               const void *beta, float *state, const int32_t *slots, int64_t pool,
                               void *y, void *stream) {
  RecurArgs a;
  const int rc = recur_check(desc, x, g, beta, true, false, &a);
  if (rc != FFT_OK) return rc;
  if (pool < 0 || (!slots && pool < desc->batch)) return FFT_ERR_INVALID_ARG;
  if (a.batch == 0 || a.tokens == 0) return FFT_OK;
  if (!y || (pool > 0 && !state)) return FFT_ERR_INVALID_ARG;
  if (off_element(y, desc->dtype) || off_element(state, FFT_ELEM_F32) ||
      off_element(slots, FFT_ELEM_F32))
    return FFT_ERR_MISALIGNED;
  a.state_out = state;
  a.slots = slots;
  a.pool = pool;
  a.y = y;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool gf = desc->gtype == FFT_ELEM_F32;
  switch (desc->dtype) {
    case FFT_ELEM_F32: return finish(launch_recur_step<float>(a, gf, st));
    case FFT_ELEM_BF16: return finish(launch_recur_step<__nv_bfloat16>(a, gf, st));
    default: return finish(launch_recur_step<__half>(a, gf, st));
  }
}

size_t fft_linear_cross_entropy_workspace_bytes(const void *x, int64_t ldx, const void *w,
                                                int64_t ldw, int64_t tokens, int64_t vocabulary,
                                                int64_t dim, int dtype, int backward) {
  XentArgs a;
  return xent_check(x, ldx, w, ldw, tokens, vocabulary, dim, dtype, &a) == FFT_OK
             ? xent_workspace_bytes(dtype, a, backward != 0)
             : 0;
}

int fft_linear_cross_entropy(const void *x, int64_t ldx, const void *w, int64_t ldw,
                             const void *targets, int target_bytes, float *loss, float *lse,
                             int64_t tokens, int64_t vocabulary, int64_t dim, int dtype,
                             void *workspace, size_t workspace_bytes, void *stream) {
  XentArgs a;
  const int rc = xent_check(x, ldx, w, ldw, tokens, vocabulary, dim, dtype, &a);
  if (rc != FFT_OK) return rc;
  if (target_bytes != 4 && target_bytes != 8) return FFT_ERR_INVALID_ARG;
  if (tokens == 0) return FFT_OK;
  if (!x || !w || !targets || !loss || !lse || !workspace ||
      workspace_bytes < xent_workspace_bytes(dtype, a, false))
    return FFT_ERR_INVALID_ARG;
  if (off_element(x, dtype) || off_element(w, dtype) || off_bytes(targets, target_bytes) ||
      off_element(loss, FFT_ELEM_F32) || off_element(lse, FFT_ELEM_F32) || misaligned(workspace))
    return FFT_ERR_MISALIGNED;
  a.targets = targets;
  a.target_bytes = target_bytes;
  a.loss = loss;
  a.lse = lse;
  return finish(launch_xent(dtype, a, workspace, static_cast<cudaStream_t>(stream)));
}

int fft_linear_cross_entropy_backward(const float *dloss, const void *x, int64_t ldx, const void *w,
                                      int64_t ldw, const void *targets, int target_bytes,
                                      const float *lse, void *dx, void *dw, int64_t tokens,
                                      int64_t vocabulary, int64_t dim, int dtype, void *workspace,
                                      size_t workspace_bytes, void *stream) {
  XentArgs a;
  const int rc = xent_check(x, ldx, w, ldw, tokens, vocabulary, dim, dtype, &a);
  if (rc != FFT_OK) return rc;
  if (target_bytes != 4 && target_bytes != 8) return FFT_ERR_INVALID_ARG;
  if (off_element(dx, dtype) || off_element(dw, dtype)) return FFT_ERR_MISALIGNED;
  if (!dx && !dw) return FFT_OK;
  if (tokens > 0) {
    if (!x || !w || !targets || !dloss || !lse || !workspace ||
        workspace_bytes < xent_workspace_bytes(dtype, a, true))
      return FFT_ERR_INVALID_ARG;
    if (off_element(x, dtype) || off_element(w, dtype) || off_bytes(targets, target_bytes) ||
        off_element(dloss, FFT_ELEM_F32) || off_element(lse, FFT_ELEM_F32) || misaligned(workspace))
      return FFT_ERR_MISALIGNED;
  }
  a.targets = targets;
  a.target_bytes = target_bytes;
  a.lse = const_cast<float *>(lse);  // read only
  a.dloss = dloss;
  a.dx = dx;
  a.dw = dw;
  return finish(launch_xent_grad(dtype, a, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
