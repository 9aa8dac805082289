// Attention over packed sequences, head dim 128.
#include "attn_packed_kernel.cuh"

namespace flex {
cudaError_t launch_packed_d128(const PackedProblem &p, const PackedParams &kp, cudaStream_t stream) {
    return launch_packed_dim<128>(p, kp, stream);
}
}  // namespace flex
