// Tensor-core backward, dK and dV of the tiles that hold a window + sinks
// mask's sinks.  Every later row keeps those columns, so that one CTA would walk
// all query tiles one after another while the other tiles' CTAs walk a window's
// (S 32768, window 1024, one head of D 128: 436 us for a backward that takes 108
// with the parts, and 76 without sinks).
// The query tiles are cut into chunks, one CTA each; the chunks' float32
// sums go to the memory of dq, which is written afterwards, and a second launch
// adds them in a fixed order and rounds once.
#include <algorithm>

#include "attn_bwd_tc_launch.cuh"
#include "bwd_internal.h"

namespace flex {
namespace {

constexpr int kSumThreads = 256;

// One thread: four neighbouring values of dv or dk.
__global__ void __launch_bounds__(kSumThreads) bwd_sum_parts_kernel(BwdTcParams p, int D) {
    const int i = (int)blockIdx.x * kSumThreads + (int)threadIdx.x;  // within [2][128][D / 4]
    const int per = 128 * D / 4, which = i / per, at = i % per * 4;
    const int own = blockIdx.y, bh = p.bh_begin + (int)blockIdx.z, row = own * 128 + at / D;
    if (which > 1 || row >= p.kv_len) return;
    const float *src = p.part + bh * p.part_stride + ((int64_t)own * p.chunks * 2 + which) * 128 * D + at;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = 0; c < p.chunks; ++c) {
        const float4 x = *reinterpret_cast<const float4 *>(src + (int64_t)c * 2 * 128 * D);
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
    }
    *reinterpret_cast<uint2 *>((which ? p.out1 : p.out0) + ((int64_t)bh * p.kv_len + row) * D + at % D) =
        make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

template <int D, int SCORE>
cudaError_t launch_parts(const CUtensorMap (&maps)[4], const BwdTcParams &kp, cudaStream_t stream) {
    using C = BwdTcCfg<D, true>;
    auto kernel = attn_bwd_tc_kernel<D, SCORE, kMaskSinks, true>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmemBytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(kp.nbh * kp.nblocks * kp.chunks), kBwdThreads, C::kSmemBytes, stream>>>(maps[0], maps[1], maps[2],
                                                                                          maps[3], kp);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const dim3 grid(2 * 128 * D / 4 / kSumThreads, (unsigned)kp.nblocks, (unsigned)kp.nbh);
    bwd_sum_parts_kernel<<<grid, kSumThreads, 0, stream>>>(kp, D);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_parts_score(const CUtensorMap (&maps)[4], const BwdTcParams &kp, int score_kind, cudaStream_t stream) {
    switch (score_kind) {
        case FLEX_SCORE_SOFTCAP:
            return launch_parts<D, FLEX_SCORE_SOFTCAP>(maps, kp, stream);
        case FLEX_SCORE_ALIBI:
            return launch_parts<D, FLEX_SCORE_ALIBI>(maps, kp, stream);
        default:
            return launch_parts<D, FLEX_SCORE_IDENTITY>(maps, kp, stream);
    }
}

}  // namespace

// The number of kv tiles, from the first, that launch_bwd_tc_dkdv_parts is to
// compute (0: none), and how it cuts them.  It pays where the walk of all query
// tiles is longer than an SM's share of all steps, those of dQ (as many) among
// them, by what the two launches take: about 10 us, a step 1 to 1.7.  Measured
// with parts and without: 32 query tiles, share 5 (window 512, four heads of D
// 128): 54 and 63 us; 64, share 36 (window 1024, eight heads): 163 and 149 us;
// 16, share 8 (window 256, sixteen heads of D 64): 49 and 41 us.
int bwd_tc_parts(const BwdTcParams &kp, int nqt, int &chunks, int &chunk_tiles) {
    constexpr int kSms = 152, kWorth = 12;
    if (mask_class(kp.mask.kind) != kMaskSinks || kp.mask.prefix <= 0) return 0;
    const int64_t tiles = ceil_blocks(std::min(kp.mask.prefix, kp.kv_len)), nbh = kp.nbh;
    const int64_t window_tiles = std::min<int64_t>(nqt, (int64_t)kp.mask.window / kBlock + 2);
    const int64_t share = nbh * ((kp.nblocks - tiles) * window_tiles + tiles * nqt) / kSms;
    if (nqt - std::max(2 * share, window_tiles) < kWorth) return 0;
    // two CTAs of parts for every SM, as far as dq's memory (2 bytes a value)
    // holds their sums (2 x 128 x D x 4 bytes each)
    int64_t n = std::min((2 * kSms + nbh * tiles - 1) / (nbh * tiles), (int64_t)kp.q_len / (4 * kBlock * tiles));
    if (n < 2) return 0;
    chunk_tiles = (int)((nqt + n - 1) / n);
    chunks = (nqt + chunk_tiles - 1) / chunk_tiles;
    return chunks < 2 ? 0 : (int)tiles;
}

cudaError_t launch_bwd_tc_dkdv_parts(const CUtensorMap (&maps)[4], const BwdTcParams &kp, int D, int score_kind,
                                     cudaStream_t stream) {
    return D == 64 ? launch_parts_score<64>(maps, kp, score_kind, stream)
                   : launch_parts_score<128>(maps, kp, score_kind, stream);
}

}  // namespace flex
