// Values of keys and values as they lie in memory, and where a packed token
// belongs: what the kernels that write and read a paged cache share.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace flex {

// Eight values as they lie in memory, and as floats.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    uint4 r;
    __device__ __forceinline__ void load(const uint16_t *src) { r = *reinterpret_cast<const uint4 *>(src); }
    __device__ __forceinline__ void unpack(float (&x)[8]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *src) {
        a = *reinterpret_cast<const float4 *>(src);
        b = *reinterpret_cast<const float4 *>(src + 4);
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};

// Packed sequences: starts[b] is the first token of sequence b, starts[n] the
// end of the last.  The sequence of a token, or -1 (before the first, behind
// the last).  Entries that do not ascend give some sequence that begins at or
// before the token.
__device__ __forceinline__ int sequence_of(const int32_t *starts, int n, int token) {
    if (n <= 0 || token < starts[0]) return -1;
    int lo = 0, hi = n;  // starts[lo] <= token
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (starts[mid] <= token)
            lo = mid;
        else
            hi = mid;
    }
    return token < starts[lo + 1] ? lo : -1;
}
// The starts for a CTA to search in: of up to kStartsHere sequences a copy in its
// shared memory, which takes one latency of device memory in place of one for each
// halving.  All threads call it, and synchronise before they search.
constexpr int kStartsHere = 127;
__device__ __forceinline__ const int32_t *stage_starts(const int32_t *starts, int n, int32_t (&here)[kStartsHere + 1]) {
    if (n > kStartsHere) return starts;
    if ((int)threadIdx.x <= n) here[threadIdx.x] = __ldg(starts + threadIdx.x);
    return here;
}

}  // namespace flex
