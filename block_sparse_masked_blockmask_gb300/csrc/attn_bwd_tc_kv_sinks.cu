// Backward, dK and dV of the kv tiles that hold a window + sinks mask's sinks.
// Every later row keeps those columns, so that one CTA would walk all query
// tiles one after another while the other tiles' CTAs walk a window's (bf16,
// S 32768, window 1024, one head of D 128: 436 us for a backward that takes 108
// with what follows, and 76 without sinks).  The query tiles are cut into
// chunks, one CTA each; the chunks' float32 sums go to the memory of dq, which is
// written afterwards, and a second launch adds them in a fixed order and rounds
// once.  Here: the rule, the sums (bf16 and fp32), and the bf16 kernel's launch.
#include <algorithm>

#include "attn_bwd_tc_launch.cuh"
#include "bwd_internal.h"

namespace flex {
namespace {

constexpr int kSumThreads = 256;

// One thread: four neighbouring values of dv or dk.
template <bool BF16>
__global__ void __launch_bounds__(kSumThreads) bwd_sum_parts_kernel(const float *part, int64_t part_stride, int chunks,
                                                                    int kv_len, int D, void *dv, void *dk) {
    const int i = (int)blockIdx.x * kSumThreads + (int)threadIdx.x;  // within [2][128][D / 4]
    const int per = kBlock * D / 4, which = i / per, at = i % per * 4;
    const int own = blockIdx.y, bh = blockIdx.z, row = own * kBlock + at / D;
    if (which > 1 || row >= kv_len) return;
    const float *src = part + bh * part_stride + ((int64_t)own * chunks * 2 + which) * kBlock * D + at;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = 0; c < chunks; ++c) {
        const float4 x = *reinterpret_cast<const float4 *>(src + (int64_t)c * 2 * kBlock * D);
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
    }
    void *out = which ? dk : dv;
    const int64_t to = ((int64_t)bh * kv_len + row) * D + at % D;
    if constexpr (BF16)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + to) =
            make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    else
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + to) = s;
}

template <int D, int SCORE>
cudaError_t launch_parts(const CUtensorMap (&maps)[4], const BwdTcParams &kp, cudaStream_t stream) {
    using C = BwdTcCfg<D, true>;
    auto kernel = attn_bwd_tc_kernel<D, SCORE, kMaskSinks, true>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmemBytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(kp.nbh * kp.nblocks * kp.chunks), kBwdThreads, C::kSmemBytes, stream>>>(maps[0], maps[1], maps[2],
                                                                                          maps[3], kp);
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

// The number of kv tiles, from the first, that are to be computed in parts (0:
// none), and how they are cut.  dq_size: bytes of one of dq's values; worth:
// steps (walked tiles) that the two launches take the time of.
// It pays where the walk of all query tiles is longer than an SM's share of all
// steps, those of dQ (as many) among them, by more than that: about 10 us, a step
// in bf16 1 to 1.7.  Measured with parts and without, bf16: 32 query tiles,
// share 5 (window 512, four heads of D 128): 54 and 63 us; 64, share 36 (window
// 1024, eight heads): 163 and 149 us; 16, share 8 (window 256, sixteen heads of
// D 64): 49 and 41 us.
int bwd_parts(const AttnProblem &p, int dq_size, int worth, int &chunks, int &chunk_tiles) {
    constexpr int kSms = 152;
    chunks = chunk_tiles = 0;
    if (mask_class(p.mask.kind) != kMaskSinks || p.mask.prefix <= 0) return 0;
    const int64_t tiles = ceil_blocks(std::min(p.mask.prefix, p.kv_len)), nbh = (int64_t)p.B * p.H, nqt = p.nqt;
    const int64_t window_tiles = std::min<int64_t>(nqt, (int64_t)p.mask.window / kBlock + 2);
    const int64_t share = nbh * ((p.nkvt - tiles) * window_tiles + tiles * nqt) / kSms;
    if (nqt - std::max(2 * share, window_tiles) < worth) return 0;
    // two CTAs of parts for every SM, as far as dq's memory holds their sums (dv
    // and dk of 128 rows in float32 each)
    const int64_t held = (int64_t)p.q_len * dq_size / (2 * kBlock * 4);
    const int64_t n = std::min((2 * kSms + nbh * tiles - 1) / (nbh * tiles), held / tiles);
    if (n < 2) return 0;
    const int len = (int)((nqt + n - 1) / n), count = (int)((nqt + len - 1) / len);
    if (count < 2) return 0;
    chunk_tiles = len;
    chunks = count;
    return (int)tiles;
}

cudaError_t launch_bwd_sum_parts(const AttnProblem &p, const float *part, int64_t part_stride, int tiles, int chunks,
                                 void *dv, void *dk, bool bf16, cudaStream_t stream) {
    // chunks >= 2 leaves fewer than 304 tiles of all heads
    const dim3 grid(2 * kBlock * p.D / 4 / kSumThreads, (unsigned)tiles, (unsigned)(p.B * p.H));
    if (bf16)
        bwd_sum_parts_kernel<true><<<grid, kSumThreads, 0, stream>>>(part, part_stride, chunks, p.kv_len, p.D, dv, dk);
    else
        bwd_sum_parts_kernel<false><<<grid, kSumThreads, 0, stream>>>(part, part_stride, chunks, p.kv_len, p.D, dv, dk);
    return cudaGetLastError();
}

cudaError_t launch_bwd_tc_dkdv_parts(const CUtensorMap (&maps)[4], const BwdTcParams &kp, int D, int score_kind,
                                     cudaStream_t stream) {
    return D == 64 ? launch_parts_score<64>(maps, kp, score_kind, stream)
                   : launch_parts_score<128>(maps, kp, score_kind, stream);
}

}  // namespace flex
