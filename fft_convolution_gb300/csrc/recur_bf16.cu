// recur_bf16.cu -- the gated linear recurrence for bfloat16 sequences (recur.cuh).
#include "recur.cuh"

namespace fftgb {
template cudaError_t launch_recur<__nv_bfloat16>(const RecurArgs &, bool, cudaStream_t);
template cudaError_t launch_recur_grad<__nv_bfloat16>(const RecurArgs &, bool, cudaStream_t);
template cudaError_t launch_recur_step<__nv_bfloat16>(const RecurArgs &, bool, cudaStream_t);
}  // namespace fftgb
