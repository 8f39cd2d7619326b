// layer_norm_bf16.cu -- bf16 instantiations of the layer normalisation
// (layer_norm.cuh).
#include "layer_norm.cuh"

namespace fftgb {

template <> cudaError_t launch_layer_norm<__nv_bfloat16>(const LayerNormArgs &a, cudaStream_t st) {
  return layer_norm_t<__nv_bfloat16>(a, st);
}
template <>
cudaError_t launch_layer_norm_grad<__nv_bfloat16>(const LayerNormGradArgs &a, cudaStream_t st) {
  return layer_norm_grad_t<__nv_bfloat16>(a, st);
}

}  // namespace fftgb
