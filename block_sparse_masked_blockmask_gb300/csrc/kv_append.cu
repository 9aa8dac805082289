// Appending keys and values to a paged cache: token t of sequence b goes to
// position cache_lens[b] + t, i.e. page page_table[b][position / page] and
// slot position % page; keys are rotated by their position on the way.
//
// A bf16 cache holds the values rounded once.  An e4m3 cache holds, for each
// (page, head), codes and one power-of-two scale s: value = code * s, with s
// the smallest power of two that keeps the page's largest magnitude within
// 448 s (e4m3's largest value).  While a page fills, its scale only grows: the
// codes already there are then divided by the growth.  Because both are powers
// of two, that is exact but for codes that fall below 2^-6 (e4m3's
// subnormals), which round once more.
//
// Bound by memory (read 2 or 4 bytes and write 1 or 2 per value).  One CTA
// owns a page of one of the two tensors for a run of heads, so the scales need
// no exchange between CTAs and no atomics in global memory: head by head it
// reads the tokens that fall on its page into registers (an item of 16 values a
// thread, or two), rotates them in float32, reduces the largest magnitude, and
// writes codes, while the next head's values are on the way.  The sines and
// cosines, which depend on (token, pair) only, are computed once per CTA into
// shared memory, to float32's accuracy: the fast sine and cosine moved 4e-5 of
// the codes of a prompt (2-norm) to a neighbour.  The rotated key is quantised
// from float32, not from a bf16 rounding of it.  Four prompts of up to 4095
// tokens (8 heads, D 128, e4m3) take 12.7 us, 4.2 TB/s: about two thirds of it
// are the instructions (a quarter of them the sines and cosines) and what the
// last CTAs leave idle.  From float32 they take 24.8 us (24.2 to a bf16 cache), half
// the rate of a copy: a block of 1024 threads, which pages of 256 tokens have, leaves
// 64 registers a thread, and the forms with two items spill, from float32 148 to
// 192 bytes a thread, from bf16 40 to 44.  A step of 32 sequences takes 3.3 us, most
// of it the launch.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "kv_internal.h"
#include "ptx.cuh"

namespace flex {
namespace {

constexpr int kMinExp = -126;  // scales are normal float32 powers of two

// Four floats to e4m3 (round to nearest even), the first in the lowest byte.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// Four e4m3 codes times f, as codes again.
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float f) {
    float x[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w >> (16 * j))));
        const __half2 h = *reinterpret_cast<const __half2 *>(&h2);
        x[2 * j] = __low2float(h) * f;
        x[2 * j + 1] = __high2float(h) * f;
    }
    return pack_e4m3x4(x[0], x[1], x[2], x[3]);
}

// The smallest power of two s with amax <= 448 s = 1.75 * 2^8 s, from the
// bits of a finite amax >= 0.
__device__ __forceinline__ float power_scale(uint32_t amax_bits) {
    int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u);
    e = max(e, kMinExp);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

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

// T: source type; E4M3: the cache's codes (else bf16); kItems: items (of 16
// values) per thread.
template <typename T, bool E4M3, int D, int kItems>
__global__ void __launch_bounds__(1024) kv_append_kernel(AppendProblem p, int heads_per_cta, int groups) {
    // cosines and sines of two pairs each: [token][quarter of an item][item],
    // so that neighbouring threads read neighbouring 16 bytes
    extern __shared__ __align__(16) float4 table[];
    __shared__ uint64_t turns[64];
    __shared__ uint32_t amax_smem[2];
    constexpr int IT = D / 16;  // items per token
    const int is_v = (int)blockIdx.z >= groups, h_first = ((int)blockIdx.z - (is_v ? groups : 0)) * heads_per_cta;
    const int b = blockIdx.y;
    const int h_last = min(h_first + heads_per_cta, p.cache.H);
    const int page = p.cache.page;
    const bool rotate = !is_v && p.inv_freq;
    const int64_t first = p.cache_lens[b];
    const int n_new = min(max(p.new_lens ? p.new_lens[b] : p.S, 0), p.S);
    if (first < 0 || n_new == 0) return;
    const int64_t slot = first / page + blockIdx.x;          // entry of the page table
    const int64_t page0 = slot * page;                       // the page's first position
    const int64_t lo = max(first, page0), hi = min(first + n_new, page0 + page);
    if (lo >= hi || slot >= p.max_pages) return;
    const int id = p.page_table[(int64_t)b * p.max_pages + slot];
    const int old_n = (int)(lo - page0);                     // tokens the page already holds
    const int n = (int)(hi - lo), total = n * IT;
    // this thread's items: where their first vectors lie, in the source (of the
    // first head) and within the page, and how far behind the second ones are
    const int64_t *st = is_v ? p.v_stride : p.k_stride;
    const T *src[kItems];
    int at[kItems], second[kItems];
    bool turned[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int i = k * (int)blockDim.x + (int)threadIdx.x, tok = i / IT, item = i % IT;
        turned[k] = rotate && item < p.rotary / 16;
        const bool half = turned[k] && p.layout == FLEX_ROPE_HALF;
        const int e = half ? item * 8 : item * 16;
        second[k] = half ? p.rotary / 2 : 8;
        src[k] = static_cast<const T *>(is_v ? p.v : p.k) + b * st[0] + h_first * st[1] + (lo + tok - first) * st[2] + e;
        at[k] = i < total ? (old_n + tok) * D + e : -1;
    }
    // a head's values, loaded one head ahead
    Raw8<T> raw[kItems][2];
    auto load = [&]() {
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            if (at[k] < 0) continue;
            raw[k][0].load(src[k]);
            raw[k][1].load(src[k] + second[k]);
            src[k] += st[1];
        }
    };
    load();
    if (rotate) {
        auto convert = [&](int i) { turns[i] = turns_per_position(p.inv_freq[i]); };
        if constexpr (kItems > 1) {  // more than 128 threads for 64 pairs at most; a loop would spill more
            if ((int)threadIdx.x < p.rotary / 2) convert((int)threadIdx.x);
        } else {
            for (int i = threadIdx.x; i < p.rotary / 2; i += blockDim.x) convert(i);
        }
        __syncthreads();
        // a thread keeps its two pairs and walks the tokens
        constexpr int kPer = 4 * IT;  // entries per token
        const int c = threadIdx.x % kPer, pair = (c % IT) * 8 + (c / IT) * 2;
        if (pair < p.rotary / 2) {
            const uint64_t t0 = turns[pair], t1 = turns[pair + 1];
            for (int tok = threadIdx.x / kPer; tok < n; tok += blockDim.x / kPer) {
                float4 w;
                sincos_at(t0, (int32_t)(lo + tok), &w.y, &w.x);
                sincos_at(t1, (int32_t)(lo + tok), &w.w, &w.z);
                w.x *= p.attention_scale;
                w.y *= p.attention_scale;
                w.z *= p.attention_scale;
                w.w *= p.attention_scale;
                table[tok * kPer + c] = w;
            }
        }
    }
    if (threadIdx.x < 2) amax_smem[threadIdx.x] = 0u;
    __syncthreads();
    if (id < 0 || id >= p.cache.num_pages) return;           // a bad page: its tokens are dropped

    float *scale_at = (is_v ? p.cache.v_scale : p.cache.k_scale) + (int64_t)id * p.cache.H;
    uint8_t *dst = (is_v ? p.cache.v : p.cache.k) + ((int64_t)id * p.cache.H + h_first) * page * D * (E4M3 ? 1 : 2);
    for (int h = h_first; h < h_last; ++h, dst += (int64_t)page * D * (E4M3 ? 1 : 2)) {
        const float old = E4M3 && old_n > 0 ? scale_at[h] : 0.f;
        float x[kItems][2][8];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            raw[k][0].unpack(x[k][0]);
            raw[k][1].unpack(x[k][1]);
        }
        if (h + 1 < h_last) load();
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            if (at[k] < 0) continue;
            if (turned[k]) {
                auto turn = [](float &a, float &z, float cs, float sn) {
                    const float a0 = a, z0 = z;
                    a = a0 * cs - z0 * sn;
                    z = z0 * cs + a0 * sn;
                };
                const int i = k * (int)blockDim.x + (int)threadIdx.x;
                const float4 *w = table + i / IT * 4 * IT + i % IT;
                if (p.layout == FLEX_ROPE_HALF) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 c = w[q * IT];
                        turn(x[k][0][2 * q], x[k][1][2 * q], c.x, c.y);
                        turn(x[k][0][2 * q + 1], x[k][1][2 * q + 1], c.z, c.w);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 c = w[q * IT];
                        float(&y)[8] = x[k][q / 2];
                        turn(y[4 * (q % 2)], y[4 * (q % 2) + 1], c.x, c.y);
                        turn(y[4 * (q % 2) + 2], y[4 * (q % 2) + 3], c.z, c.w);
                    }
                }
            }
            if constexpr (E4M3) {
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmax3(top, fabsf(x[k][0][j]), fabsf(x[k][1][j]));  // NaN: passed over
            }
        }
        float inv = 1.f;
        if constexpr (E4M3) {
            // two words take turns: one is cleared for the next head while the other is in use
            uint32_t *amax = &amax_smem[(h - h_first) & 1];
            const uint32_t top_bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
            if (threadIdx.x % 32 == 0) atomicMax(amax, top_bits);
            __syncthreads();
            uint32_t most = *amax;
            if (most == 0x7F800000u) {
                // an infinity among the values: it becomes NaN and has no part in the scale
                __syncthreads();
                if (threadIdx.x == 0) *amax = 0u;
                __syncthreads();
                uint32_t finite = 0u;
#pragma unroll
                for (int k = 0; k < kItems; ++k)
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        if (at[k] < 0) continue;
                        float &y = x[k][j / 8][j % 8];
                        const uint32_t w = __float_as_uint(y) & 0x7FFFFFFFu;
                        if (w >= 0x7F800000u)
                            y = __uint_as_float(0x7FC00000u);
                        else
                            finite = max(finite, w);
                    }
                finite = __reduce_max_sync(0xffffffffu, finite);
                if (threadIdx.x % 32 == 0) atomicMax(amax, finite);
                __syncthreads();
                most = *amax;
            }
            const float want = power_scale(most);
            const float now = old > want ? old : want;
            if (threadIdx.x == 0) {
                scale_at[h] = now;
                amax_smem[(h - h_first + 1) & 1] = 0u;
            }
            if (old_n > 0 && now != old) {
                const float f = old / now;
                uint4 *codes = reinterpret_cast<uint4 *>(dst);
                for (int i = threadIdx.x; i < old_n * D / 16; i += blockDim.x) {
                    uint4 w = codes[i];
                    w.x = rescale_e4m3x4(w.x, f);
                    w.y = rescale_e4m3x4(w.y, f);
                    w.z = rescale_e4m3x4(w.z, f);
                    w.w = rescale_e4m3x4(w.w, f);
                    codes[i] = w;
                }
            }
            inv = 1.f / now;  // exact for a power of two, which `now` is unless the page came with another scale
            if (h + 1 < h_last) __syncthreads();  // the cleared word, before the next head's maxima
        }
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            if (at[k] < 0) continue;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float(&y)[8] = x[k][u];
                const int e = at[k] + (u ? second[k] : 0);
                if constexpr (E4M3)
                    *reinterpret_cast<uint2 *>(dst + e) =
                        make_uint2(pack_e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                                   pack_e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
                else
                    *reinterpret_cast<uint4 *>(dst + 2 * e) =
                        make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                   pack_bf16x2(y[6], y[7]));
            }
        }
    }
}

template <typename T, bool E4M3, int D, int kItems>
cudaError_t launch_append(const AppendProblem &p, cudaStream_t stream) {
    const int page = p.cache.page;
    // threads for the tokens that can fall on one page
    const int most = (p.S < page ? p.S : page) * (D / 16);
    int threads = (most + kItems - 1) / kItems;
    threads = (threads + 31) / 32 * 32;
    // pages that S tokens can touch, starting anywhere in one
    const int64_t pages = ((int64_t)p.S + page - 2) / page + 1;
    const int64_t slots = pages < p.max_pages ? pages : p.max_pages;
    // heads per CTA: up to 8 share the sines and cosines, as long as that
    // leaves six CTAs for every SM (2 heads instead of 4 at 528 pages of 8 heads
    // and two tensors: 16.2 us for 14.0; 4 instead of 2 at 204 of 16: 5.0 for 4.6)
    int heads = 8;
    while (heads > 1 && slots * p.B * 2 * ((p.cache.H + heads - 1) / heads) < 6 * 152) heads /= 2;
    // the CTAs of the keys, which have the sines and cosines to do, come first,
    // and those of the values fill in behind them (alternating: 16.0 us for 13.9)
    const int groups = (p.cache.H + heads - 1) / heads;
    const dim3 grid((unsigned)slots, p.B, 2u * groups);
    const int smem = p.inv_freq ? (p.S < page ? p.S : page) * D * 4 : 0;  // one (cosine, sine) per pair of a head
    auto kernel = kv_append_kernel<T, E4M3, D, kItems>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    kernel<<<grid, threads, smem, stream>>>(p, heads, groups);
    return cudaGetLastError();
}

template <typename T, bool E4M3>
cudaError_t launch_append_d(const AppendProblem &p, cudaStream_t stream) {
    // one item a thread while that makes at most 256 threads: two halve what a
    // head costs beside its values, which pays where there are warps enough
    // (pages of 512 items: 14.0 us for 18.0 with one; of 64: 6.9 for 4.6)
    const int items = (p.S < p.cache.page ? p.S : p.cache.page) * (p.cache.D / 16);
    if (p.cache.D == 64)
        return items <= 256 ? launch_append<T, E4M3, 64, 1>(p, stream) : launch_append<T, E4M3, 64, 2>(p, stream);
    return items <= 256 ? launch_append<T, E4M3, 128, 1>(p, stream) : launch_append<T, E4M3, 128, 2>(p, stream);
}

}  // namespace

cudaError_t launch_kv_append(const AppendProblem &p, int src_dtype, int cache_dtype, cudaStream_t stream) {
    const bool e4m3 = cache_dtype == FLEX_DTYPE_E4M3;
    if (src_dtype == FLEX_DTYPE_BF16)
        return e4m3 ? launch_append_d<uint16_t, true>(p, stream) : launch_append_d<uint16_t, false>(p, stream);
    return e4m3 ? launch_append_d<float, true>(p, stream) : launch_append_d<float, false>(p, stream);
}

}  // namespace flex
