// recur_f32.cu -- the gated linear recurrence for float sequences (recur.cuh).
#include "recur.cuh"

namespace fftgb {
template cudaError_t launch_recur<float>(const RecurArgs &, bool, cudaStream_t);
template cudaError_t launch_recur_grad<float>(const RecurArgs &, bool, cudaStream_t);
template cudaError_t launch_recur_step<float>(const RecurArgs &, bool, cudaStream_t);
}  // namespace fftgb
