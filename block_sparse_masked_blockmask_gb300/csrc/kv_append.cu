// Appending [B, H, S, D] keys and values to a paged cache of bf16 or e4m3.
#include "kv_append_kernel.cuh"

namespace flex {

cudaError_t launch_kv_append(const AppendProblem &p, int src_dtype, int cache_dtype, cudaStream_t stream) {
    return p.starts ? launch_kv_append_packed(p, src_dtype, cache_dtype, stream)
                    : launch_append_typed<false>(p, src_dtype, cache_dtype, stream);
}

}  // namespace flex
