// delta_launch.cuh -- the launches of the gated delta rule over whole
// sequences, for one element type.
#pragma once

#include "delta_back.cuh"
#include "delta_grad.cuh"

namespace fftgb {

// The plan of the chunks, made by a small kernel for packed sequences.
template <typename T>
cudaError_t delta_make_plan(const DeltaArgs &a, const DeltaGradArgs *g, const DeltaLayout &w,
                            char *ws, DeltaPlan &plan, cudaStream_t st) {
  plan.row0 = plan.chunk0 = nullptr;
  plan.chunks_max = w.chunks;
  plan.per_seq = (int)((a.tokens + kChunk - 1) / kChunk);
  if (!a.offsets) return cudaSuccess;
  int *row0 = reinterpret_cast<int *>(ws + w.row0), *chunk0 = reinterpret_cast<int *>(ws + w.chunk0);
  plan.row0 = row0;
  plan.chunk0 = chunk0;
  return launch_delta_plan(a.offsets, a.batch, a.tokens, row0, chunk0, delta_clear(a, g, sizeof(T)),
                           st);
}

template <typename T, int DK, bool GRAD>
cudaError_t delta_prep_t(const DeltaArgs &a, const DeltaPlan &plan, char *kq, char *images,
                         char *back, int *status, cudaStream_t st) {
  static DeviceOnce once;
  const void *kern = (const void *)delta_prep_kernel<T, DK, GRAD>;
  cudaError_t e = smem_limit_once(kern, prep_smem<T, DK>(), once);
  if (e != cudaSuccess) return e;
  const long long blocks = plan.chunks_max * a.kheads;
  if (blocks == 0) return cudaSuccess;
  delta_prep_kernel<T, DK, GRAD>
      <<<(unsigned)blocks, kPrepThreads, prep_smem<T, DK>(), st>>>(a, plan, kq, images, back,
                                                                       status);
  return cudaGetLastError();
}

// Whether rows of 128 columns (fewer at the end) can go by bulk copies.
template <typename T> bool delta_staged(const DeltaArgs &a, const void *in, const DeltaStride &s,
                                        const void *out) {
  return sizeof(T) == 2 && a.dv % 8 == 0 && vec_rows<T>(in, s) && ((uintptr_t)out & 15u) == 0;
}

template <typename T, int DK, bool STAGED>
cudaError_t delta_scan_t(const DeltaArgs &a, const DeltaPlan &plan, const char *kq,
                         const char *images, int *status, cudaStream_t st) {
  constexpr size_t smem = scan_smem(DK, Terms<T>::value, STAGED);
  static DeviceOnce once;
  auto kern = delta_scan_kernel<T, DK, STAGED>;
  cudaError_t e = smem_limit_once((const void *)kern, smem, once);
  if (e != cudaSuccess) return e;
  const long long blocks = a.batch * a.vheads * ((a.dv + 127) / 128);
  kern<<<(unsigned)blocks, kScanThreads, smem, st>>>(a, plan, kq, images, status);
  return cudaGetLastError();
}

template <typename T, int DK>
cudaError_t delta_forward_t(const DeltaArgs &a, char *ws, cudaStream_t st) {
  int *status = device_status_word();
  if (!status) return cudaErrorInvalidDevice;
  const DeltaLayout w(a, a.offsets != nullptr, false);
  DeltaPlan plan;
  cudaError_t e = delta_make_plan<T>(a, nullptr, w, ws, plan, st);
  if (e == cudaSuccess) e = delta_prep_t<T, DK, false>(a, plan, ws + w.kq, ws + w.images, nullptr, status, st);
  if (e != cudaSuccess) return e;
  if constexpr (sizeof(T) == 2)
    if (delta_staged<T>(a, a.v, a.sv, a.o))
      return delta_scan_t<T, DK, true>(a, plan, ws + w.kq, ws + w.images, status, st);
  return delta_scan_t<T, DK, false>(a, plan, ws + w.kq, ws + w.images, status, st);
}

template <typename T, int DK, bool STAGED>
cudaError_t delta_scans_t(const DeltaArgs &a, const DeltaGradArgs &g, const DeltaPlan &plan,
                          const char *kq, const char *images, const char *back, char *states,
                          char *dstates, char *es, char *fs, char *os, float *scales, int *status,
                          cudaStream_t st) {
  constexpr size_t smem = scan_smem(DK, Terms<T>::value, STAGED);
  static DeviceOnce once;
  auto kern = delta_scans_kernel<T, DK, STAGED>;
  cudaError_t e = smem_limit_once((const void *)kern, smem, once);
  if (e != cudaSuccess) return e;
  const long long blocks = 2 * a.batch * a.vheads * ((a.dv + 127) / 128);
  kern<<<(unsigned)blocks, kScanThreads, smem, st>>>(a, g, plan, kq, images, back, states, dstates,
                                                     es, fs, os, scales, status);
  return cudaGetLastError();
}
template <typename T> bool delta_scans_staged(const DeltaArgs &a, const DeltaGradArgs &g) {
  return delta_staged<T>(a, a.v, a.sv, a.o) &&
         (((uintptr_t)g.dout | (uintptr_t)g.dv) & 15u) == 0;
}

template <typename T, int DK, bool MULTI>
cudaError_t delta_grad_t(const DeltaArgs &a, const DeltaGradArgs &g, const DeltaPlan &plan,
                         const char *kq, const char *back, const char *states,
                         const char *dstates, char *es, char *fs, const char *os,
                         const float *scales, int *status, cudaStream_t st) {
  constexpr size_t smem = grad_smem(DK, Terms<T>::value);
  static DeviceOnce once;
  auto kern = delta_grad_kernel<T, DK, MULTI>;
  cudaError_t e = smem_limit_once((const void *)kern, smem, once);
  const long long chunks = plan.chunks_max;
  if (e != cudaSuccess || chunks == 0) return e;
  const long long items = chunks * a.vheads;
  const int blocks = (int)(items < sm_count() ? items : sm_count());
  const bool partial = a.vheads > a.kheads;
  kern<<<blocks, kGradThreads, smem, st>>>(a, g, plan, kq, back, states, dstates, es, fs, os,
                                           scales, partial, status);
  e = cudaGetLastError();
  if (e != cudaSuccess || !partial) return e;
  delta_grad_sum_kernel<T, DK><<<dim3((unsigned)(chunks * a.kheads), 2), 256, 0, st>>>(
      a, g, plan, reinterpret_cast<const float *>(es), reinterpret_cast<const float *>(fs));
  return cudaGetLastError();
}

template <typename T, int DK>
cudaError_t delta_backward_t(const DeltaArgs &a, const DeltaGradArgs &g, char *ws,
                             cudaStream_t st) {
  int *status = device_status_word();
  if (!status) return cudaErrorInvalidDevice;
  const DeltaLayout w(a, a.offsets != nullptr, true);
  char *kq = ws + w.kq, *images = ws + w.images, *back = ws + w.back;
  char *states = ws + w.state, *dstates = ws + w.dstate, *es = ws + w.e, *fs = ws + w.f, *os = ws + w.o;
  float *scales = reinterpret_cast<float *>(ws + w.scales);
  DeltaPlan plan;
  cudaError_t e = delta_make_plan<T>(a, &g, w, ws, plan, st);
  if (e == cudaSuccess) e = delta_prep_t<T, DK, true>(a, plan, kq, images, back, status, st);
  if (e != cudaSuccess) return e;
  auto scans = delta_scans_t<T, DK, false>;
  if constexpr (sizeof(T) == 2)
    if (delta_scans_staged<T>(a, g)) scans = delta_scans_t<T, DK, true>;
  e = scans(a, g, plan, kq, images, back, states, dstates, es, fs, os, scales, status, st);
  if (e != cudaSuccess) return e;
  auto grad = a.dv <= 128 ? delta_grad_t<T, DK, false> : delta_grad_t<T, DK, true>;
  return grad(a, g, plan, kq, back, states, dstates, es, fs, os, scales, status, st);
}

}  // namespace fftgb
