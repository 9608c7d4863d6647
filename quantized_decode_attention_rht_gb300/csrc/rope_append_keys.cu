// Large rotary appends: the key side's instances (rope_append_large.cuh).
#include "rope_append_large.cuh"

namespace kvq {
cudaError_t launch_append_keys(const LargeParams& p, int head_dim, int sms, cudaStream_t stream) {
  return launch_large_dim<true>(p, head_dim, sms, stream);
}
}  // namespace kvq
