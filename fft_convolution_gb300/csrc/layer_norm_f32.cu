// layer_norm_f32.cu -- f32 instantiations of the layer normalisation
// (layer_norm.cuh),
// plus its host-side sizing.
#include "layer_norm.cuh"

namespace fftgb {

int layer_norm_partials(int dtype, long long rows, int dim) {
  if (dtype == FFT_ELEM_F64 || dim > kNormRegMax)
    return (int)(rows < kLongParts ? rows : kLongParts);
  return (int)norm_grid(rows, dim) * norm_groups(dim);
}

template <> cudaError_t launch_layer_norm<float>(const LayerNormArgs &a, cudaStream_t st) {
  return layer_norm_t<float>(a, st);
}
template <>
cudaError_t launch_layer_norm_grad<float>(const LayerNormGradArgs &a, cudaStream_t st) {
  return layer_norm_grad_t<float>(a, st);
}

}  // namespace fftgb
