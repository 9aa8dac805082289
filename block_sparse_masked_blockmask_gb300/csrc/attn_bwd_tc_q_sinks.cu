// Tensor-core backward, dQ under window + sinks masks (a row keeps two
// intervals; dK and dV, whose columns keep one, run as interval masks).
#include <algorithm>

#include "attn_bwd_tc_launch.cuh"
#include "bwd_internal.h"

namespace flex {
cudaError_t launch_bwd_tc_dq_sinks(const CUtensorMap (&maps)[4], const BwdTcParams &kp, int D, int score_kind,
                                   cudaStream_t stream) {
    return D == 64 ? launch_bwd_tc_score<64, kMaskSinks, false>(maps, kp, score_kind, stream)
                   : launch_bwd_tc_score<128, kMaskSinks, false>(maps, kp, score_kind, stream);
}
}  // namespace flex
