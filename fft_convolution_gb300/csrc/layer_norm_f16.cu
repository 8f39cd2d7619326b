// layer_norm_f16.cu -- f16 instantiations of the layer normalisation
// (layer_norm.cuh).
#include "layer_norm.cuh"

namespace fftgb {

template <> cudaError_t launch_layer_norm<__half>(const LayerNormArgs &a, cudaStream_t st) {
  return layer_norm_t<__half>(a, st);
}
template <>
cudaError_t launch_layer_norm_grad<__half>(const LayerNormGradArgs &a, cudaStream_t st) {
  return layer_norm_grad_t<__half>(a, st);
}

}  // namespace fftgb
