// delta_f32.cu -- f32 instantiations of the gated delta rule over whole
// sequences (delta_launch.cuh).
#include "delta_launch.cuh"

namespace fftgb {

template <>
cudaError_t launch_delta<float>(const DeltaArgs &a, void *workspace, cudaStream_t st) {
  char *ws = static_cast<char *>(workspace);
  return a.dk <= 64 ? delta_forward_t<float, 64>(a, ws, st) : delta_forward_t<float, 128>(a, ws, st);
}

template <>
cudaError_t launch_delta_grad<float>(const DeltaArgs &a, const DeltaGradArgs &g, void *workspace,
                                cudaStream_t st) {
  char *ws = static_cast<char *>(workspace);
  return a.dk <= 64 ? delta_backward_t<float, 64>(a, g, ws, st)
                    : delta_backward_t<float, 128>(a, g, ws, st);
}

}  // namespace fftgb
