// recur_f16.cu -- the gated linear recurrence for half sequences (recur.cuh).
#include "recur.cuh"

namespace fftgb {
template cudaError_t launch_recur<__half>(const RecurArgs &, bool, cudaStream_t);
template cudaError_t launch_recur_grad<__half>(const RecurArgs &, bool, cudaStream_t);
template cudaError_t launch_recur_step<__half>(const RecurArgs &, bool, cudaStream_t);
}  // namespace fftgb
