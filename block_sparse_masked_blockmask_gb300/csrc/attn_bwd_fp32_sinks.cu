// The fp32 tensor-core backward under window + sinks masks (compiled apart so
// that the instantiations build in parallel).
#include "attn_bwd_fp32_tc.cuh"

namespace flex {
template cudaError_t launch_bwd_fp32_tc_dkdv<true>(const AttnProblem &, const BwdF32TcArgs &, int, cudaStream_t);
template cudaError_t launch_bwd_fp32_tc_dq<true>(const AttnProblem &, const BwdF32TcArgs &, cudaStream_t);
}  // namespace flex
