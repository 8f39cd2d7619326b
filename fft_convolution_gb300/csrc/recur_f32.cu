// recur_f32.cu -- the gated linear recurrence for float sequences (recur.cuh).
#include "recur.cuh"

namespace fftgb {
// From this many packed sequences on a kernel of its own finds their rows (5 us);
// below, each block looks through the offsets before its own, four at most per thread.
size_t recur_workspace_bytes(long long batch, bool packed) {
  return packed && batch > 1024 ? 2 * (size_t)(batch + 1) * sizeof(int) : 0;
}
template cudaError_t launch_recur<float>(const RecurArgs &, bool, cudaStream_t);
template cudaError_t launch_recur_grad<float>(const RecurArgs &, bool, cudaStream_t);
template cudaError_t launch_recur_step<float>(const RecurArgs &, bool, cudaStream_t);
}  // namespace fftgb
