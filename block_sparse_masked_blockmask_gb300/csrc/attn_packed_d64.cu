// Attention over packed sequences, head dim 64.
#include "attn_packed_kernel.cuh"

namespace flex {
cudaError_t launch_packed_d64(const PackedProblem &p, const PackedParams &kp, cudaStream_t stream) {
    return launch_packed_dim<64>(p, kp, stream);
}
}  // namespace flex
