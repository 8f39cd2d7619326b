// layer_norm_f64.cu -- f64 instantiations of the layer normalisation
// (layer_norm.cuh).
#include "layer_norm.cuh"

namespace fftgb {

template <> cudaError_t launch_layer_norm<double>(const LayerNormArgs &a, cudaStream_t st) {
  return layer_norm_t<double>(a, st);
}
template <>
cudaError_t launch_layer_norm_grad<double>(const LayerNormGradArgs &a, cudaStream_t st) {
  return layer_norm_grad_t<double>(a, st);
}

}  // namespace fftgb
