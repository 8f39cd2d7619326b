// delta_bf16.cu -- bf16 instantiations of the gated delta rule over whole
// sequences (delta_launch.cuh).
#include "delta_launch.cuh"

namespace fftgb {

template <>
cudaError_t launch_delta<__nv_bfloat16>(const DeltaArgs &a, void *workspace, cudaStream_t st) {
  char *ws = static_cast<char *>(workspace);
  return a.dk <= 64 ? delta_forward_t<__nv_bfloat16, 64>(a, ws, st) : delta_forward_t<__nv_bfloat16, 128>(a, ws, st);
}

template <>
cudaError_t launch_delta_grad<__nv_bfloat16>(const DeltaArgs &a, const DeltaGradArgs &g, void *workspace,
                                cudaStream_t st) {
  char *ws = static_cast<char *>(workspace);
  return a.dk <= 64 ? delta_backward_t<__nv_bfloat16, 64>(a, g, ws, st)
                    : delta_backward_t<__nv_bfloat16, 128>(a, g, ws, st);
}

}  // namespace fftgb
