// Rotary positions: pairs of a head's values turned by an angle that grows
// with the token's position,
//   (x0, x1) -> a (x0 cos - x1 sin, x1 cos + x0 sin),  angle = position * inv_freq[i],
// for q and k in one launch; backward is the same with the angle negated (the
// matrix is a times a rotation, its transpose a times the rotation back).
//
// Bound by memory: every value is read once and written once.  The angle and
// its sine and cosine depend on (token, pair) only, so a thread keeps them in
// registers for one item (two 16-byte vectors: the two halves of eight pairs,
// or four in fp32) of one token and walks the heads of both tensors with them.
// Rotating a bf16 head costs two loads, two stores and ~60 other instructions
// per thread; a sine and cosine cost ~40, which four heads or more per thread hide.
// q and k of B2 H32 S16384 D128 in bf16 take 163 us, 6.6 TB/s: 97% of the rate
// of a copy.  A step of 16 sequences (40 heads each) takes 3.1 us, of which the
// launch is most.
// Frequencies are converted to fixed-point turns once per CTA, by a product of
// whole numbers that a token's heads do not repeat.
#include <cuda_bf16.h>

#include "kv_internal.h"
#include "ptx.cuh"

namespace flex {
namespace {

constexpr int kRopeThreads = 256;

// A 16-byte vector as floats, and back (bf16: 8 values; fp32: 4).
template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &r, float (&x)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 &r, float (&x)[4]) {
        x[0] = __uint_as_float(r.x);
        x[1] = __uint_as_float(r.y);
        x[2] = __uint_as_float(r.z);
        x[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeProblem p, int heads_per_cta) {
    constexpr int V = Vec<T>::N;
    constexpr int UN = 4;  // heads in flight
    __shared__ uint64_t turns[64];
    for (int i = threadIdx.x; i < p.rotary / 2; i += kRopeThreads) turns[i] = turns_per_position(p.inv_freq[i]);
    __syncthreads();
    const int items = p.D / (2 * V);
    const int64_t at = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
    const int item = (int)(at % items);
    const int64_t token = at / items;
    if (token >= (int64_t)p.B * p.S) return;
    const int b = (int)(token / p.S), s = (int)(token % p.S);
    const bool turned = item < p.rotary / (2 * V);
    // the item's two vectors within the head
    const int e0 = LAYOUT == FLEX_ROPE_HALF && turned ? item * V : item * 2 * V;
    const int e1 = LAYOUT == FLEX_ROPE_HALF && turned ? p.rotary / 2 + item * V : e0 + V;
    float c[V], n[V];
    if (turned) {
        const int pos = p.positions ? p.positions[token] : s;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            sincos_at(turns[item * V + j], pos, &n[j], &c[j]);
            c[j] *= p.attention_scale;
            n[j] *= p.attention_scale * p.direction;
        }
    }
    const int total = p.heads[0] + p.heads[1];
    const int h0 = blockIdx.y * heads_per_cta, h1 = min(h0 + heads_per_cta, total);
    for (int base = h0; base < h1; base += UN) {
        uint4 r0[UN], r1[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            if (base + u >= h1) continue;
            const int w = base + u >= p.heads[0], h = base + u - (w ? p.heads[0] : 0);
            const T *src = static_cast<const T *>(p.in[w]) + b * p.in_stride[w][0] + h * p.in_stride[w][1] +
                           s * p.in_stride[w][2];
            r0[u] = *reinterpret_cast<const uint4 *>(src + e0);
            r1[u] = *reinterpret_cast<const uint4 *>(src + e1);
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            if (base + u >= h1) continue;
            const int w = base + u >= p.heads[0], h = base + u - (w ? p.heads[0] : 0);
            T *dst = static_cast<T *>(p.out[w]) + b * p.out_stride[w][0] + h * p.out_stride[w][1] +
                     s * p.out_stride[w][2];
            if (turned) {
                float x0[V], x1[V];
                Vec<T>::unpack(r0[u], x0);
                Vec<T>::unpack(r1[u], x1);
                if constexpr (LAYOUT == FLEX_ROPE_HALF) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float a = x0[j], z = x1[j];
                        x0[j] = a * c[j] - z * n[j];
                        x1[j] = z * c[j] + a * n[j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) {
                        float a = x0[2 * j], z = x0[2 * j + 1];
                        x0[2 * j] = a * c[j] - z * n[j];
                        x0[2 * j + 1] = z * c[j] + a * n[j];
                        a = x1[2 * j];
                        z = x1[2 * j + 1];
                        x1[2 * j] = a * c[V / 2 + j] - z * n[V / 2 + j];
                        x1[2 * j + 1] = z * c[V / 2 + j] + a * n[V / 2 + j];
                    }
                }
                r0[u] = Vec<T>::pack(x0);
                r1[u] = Vec<T>::pack(x1);
            }
            *reinterpret_cast<uint4 *>(dst + e0) = r0[u];
            *reinterpret_cast<uint4 *>(dst + e1) = r1[u];
        }
    }
}

template <typename T>
cudaError_t launch_rope_typed(const RopeProblem &p, cudaStream_t stream) {
    const int64_t threads = (int64_t)p.B * p.S * (p.D / (2 * Vec<T>::N));
    const int64_t ctas = (threads + kRopeThreads - 1) / kRopeThreads;
    const int total = p.heads[0] + p.heads[1];
    // Heads per CTA: 16, so that the angles are shared, unless that leaves
    // fewer than four CTAs for every SM; four are loaded at a time
    int per = 16;
    while (per > 4 && ctas * ((total + per - 1) / per) < 4 * 152) per /= 2;
    const dim3 grid((unsigned)ctas, (unsigned)((total + per - 1) / per));
    if (p.layout == FLEX_ROPE_HALF)
        rope_kernel<T, FLEX_ROPE_HALF><<<grid, kRopeThreads, 0, stream>>>(p, per);
    else
        rope_kernel<T, FLEX_ROPE_INTERLEAVED><<<grid, kRopeThreads, 0, stream>>>(p, per);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeProblem &p, int dtype, cudaStream_t stream) {
    return dtype == FLEX_DTYPE_BF16 ? launch_rope_typed<uint16_t>(p, stream) : launch_rope_typed<float>(p, stream);
}

}  // namespace flex
