// Internal declarations shared by the CUDA translation units of the library:
// the device-side mask description, the mask_mod predicate, the kernel
// launchers called by the C-ABI layer, and the per-device workspace.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>
#include <cuda.h>

#include "../../include/flexattn.h"

namespace flex {

constexpr int kBlock = 128;         // compute tile (128 x 128); BlockMask blocks of other sizes map onto it
constexpr int kMaxKvBlocks = 1024;  // kv tiles (of 128) per row the kernels stage on chip
constexpr int kMinListBlock = 16, kMaxListBlock = 1024;  // BlockMask block sizes: powers of two in this range

__host__ __device__ constexpr bool valid_block_size(int b) {
    return b >= kMinListBlock && b <= kMaxListBlock && (b & (b - 1)) == 0;
}
// Blocks of size bs along a length (the last one may reach past it).
__host__ __device__ constexpr int ceil_div(int64_t len, int bs) { return (int)((len + bs - 1) / bs); }

// mask_mod as the kernels see it.
struct MaskDesc {
    int32_t kind;
    int32_t window;
    int32_t prefix;             // causal + prefix: inclusive bound; window + sinks: first tokens that stay visible
    int32_t doc_len;            // row length of doc_ids (== q_len == kv_len)
    const int32_t *doc_ids;     // [B, doc_len]
    int32_t q_len, kv_len;      // positions at or past these are padding: masked
};

// Tiles along a length: the last one may reach past it (padding, masked).
__host__ __device__ constexpr int ceil_blocks(int64_t len) { return (int)((len + kBlock - 1) / kBlock); }

// mask_mod(b, h, q, kv) for the enumerated kinds but window + sinks (mask_keep
// below).  No kind depends on h.
__host__ __device__ __forceinline__ bool mask_mod(const MaskDesc &m, int b, int q, int kv) {
    switch (m.kind) {
        case FLEX_MASK_CAUSAL:
            return q >= kv;
        case FLEX_MASK_SLIDING_WINDOW:
            return q >= kv && q - kv < m.window;
        case FLEX_MASK_CAUSAL_PREFIX:
            return (q <= m.prefix && kv <= m.prefix) || q >= kv;
        case FLEX_MASK_DOCUMENT:
            return q >= kv && m.doc_ids[(int64_t)b * m.doc_len + q] == m.doc_ids[(int64_t)b * m.doc_len + kv];
        default:
            return true;
    }
}

// The interval kinds keep, for a fixed row q, exactly the kv in [lo, hi].
// Returns false for kinds whose kept set is not an interval (document, window
// + sinks).
__host__ __device__ __forceinline__ bool mask_row_interval(const MaskDesc &m, int q, int &lo, int &hi) {
    switch (m.kind) {
        case FLEX_MASK_CAUSAL:
            lo = 0;
            hi = q;
            return true;
        case FLEX_MASK_SLIDING_WINDOW:
            lo = q - m.window + 1;
            hi = q;
            return true;
        case FLEX_MASK_CAUSAL_PREFIX:
            lo = 0;
            hi = q <= m.prefix ? m.prefix : q;
            return true;
        case FLEX_MASK_ALL:
            lo = 0;
            hi = 0x7fffffff;
            return true;
        default:
            return false;
    }
}

// The window + sinks kind keeps two intervals per row, [0, sink_hi] and
// [lo, q].  Once the window reaches down to the sinks they are one,
// [0, q] (sink_hi is then q, and lo 0).
__host__ __device__ __forceinline__ void mask_row_sinks(const MaskDesc &m, int q, int &sink_hi, int &lo) {
    lo = q - m.window + 1 > 0 ? q - m.window + 1 : 0;
    sink_hi = m.prefix - 1 < q ? m.prefix - 1 : q;
    if (lo <= sink_hi + 1) {
        lo = 0;
        sink_hi = q;
    }
}

// mask_mod in kernels compiled apart for window + sinks masks: one more case
// in the switch above made the fp32 backward 6% slower for every kind.
template <bool SINKS>
__host__ __device__ __forceinline__ bool mask_keep(const MaskDesc &m, int b, int q, int kv) {
    if constexpr (SINKS) return q >= kv && (q - kv < m.window || kv < m.prefix);
    return mask_mod(m, b, q, kv);
}

// Mask classes the attention kernels are compiled for: interval kinds, the
// document kind, and window + sinks.
enum : int { kMaskInterval = 0, kMaskDocument = 1, kMaskSinks = 2 };
__host__ __device__ constexpr int mask_class(int kind) {
    return kind == FLEX_MASK_DOCUMENT ? kMaskDocument : kind == FLEX_MASK_WINDOW_SINKS ? kMaskSinks : kMaskInterval;
}

// Problem description handed from the C-ABI layer to the attention launchers.
struct AttnProblem {
    int B, H, q_len, kv_len, D;
    int q_block, kv_block, nqb, nkvb;                // BlockMask granularity: block sizes, blocks per row/column
    int nqt, nkvt;                                   // 128-tiles along q and kv
    int bh_begin, bh_count;                          // the (b, h) pairs b * H + h in [bh_begin, +bh_count) are computed
    int64_t q_stride[4], k_stride[4], v_stride[4];  // elements
    const void *q, *k, *v;
    void *out;                                       // contiguous [B,H,q_len,D]
    float *lse;                                      // contiguous [B,H,q_len]
    const int32_t *kv_num, *kv_idx, *full_num, *full_idx;
    MaskDesc mask;
    int score_kind;
    float score_param;
    float scale;
    int prescale;                                    // PRESCALE_QK: Q is scaled (rounded to its dtype) before QK^T
    float *row_max;                                  // OUTPUT_MAX: contiguous [B,H,q_len] or null
    int *status;                                     // device status word
};

// Launchers (return a cudaError_t from the launch).
cudaError_t launch_block_mask(const MaskDesc &mask, int B, int H, int q_len, int kv_len, int q_block, int kv_block,
                              int32_t *kv_num, int32_t *kv_idx, int32_t *full_num, int32_t *full_idx,
                              cudaStream_t stream);
cudaError_t launch_attn_fp32(const AttnProblem &p, cudaStream_t stream);
cudaError_t launch_attn_bf16(const AttnProblem &p, cudaStream_t stream);

// TMA tensor map of a bf16 [B, H, S, D] tensor with element strides st
// (st[3] == 1): 64 x 128 boxes (head dims x rows), 128-byte swizzle.
bool make_bf16_tile_map(CUtensorMap *map, const void *base, int B, int H, int S, int D, const int64_t st[4]);

// TMA tensor map of a 3-D view (innermost extent first; strides in bytes).
bool make_tile_map_3d(CUtensorMap *map, const void *base, CUtensorMapDataType type, const uint64_t (&dims)[3],
                      const uint64_t (&strides)[2], const uint32_t (&box)[3], CUtensorMapSwizzle swizzle);

cudaError_t launch_wait_timeout_selftest(int *status, uint64_t limit_ns, cudaStream_t stream);

// Argument checks shared by the C-ABI layer's files: a [B, H, S, D] tensor of
// the given type and shape with 16-byte aligned base and strides, inner stride
// 1; and the parameters of the windowed mask kinds.
int check_tensor(const flex_tensor *t, int dtype, int64_t B, int64_t H, int64_t S, int64_t D);
bool valid_window(int kind, const flex_mask_params &prm);

// The per-device workspace holding the status word (allocated once per device).
int *device_status_word(int *err);

// Status codes a kernel writes into the status word.
constexpr int kDeviceTimeout = 1;

}  // namespace flex
