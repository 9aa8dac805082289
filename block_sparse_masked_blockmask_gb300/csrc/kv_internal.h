// Internal declarations of the rotary positions and the paged key/value
// cache: problem descriptions handed from the C-ABI layer to the launchers,
// and the arithmetic that both the rotation kernel and the append share.
#pragma once

#include "flex_internal.h"

namespace flex {

struct RopeProblem {
    int B, S, D;
    int heads[2];                    // heads of the two tensors (0: no second tensor)
    const void *in[2];
    void *out[2];
    int64_t in_stride[2][3], out_stride[2][3];  // b, h, s (elements)
    const double *inv_freq;          // radians per position, rotary / 2 of them
    const int32_t *positions;        // [B, S], or null: 0 .. S - 1
    int rotary, layout;
    float attention_scale;
    float direction;                 // +1 rotates forward, -1 back
};

struct KvCache {
    int num_pages, H, page, D, page_shift;
    uint8_t *k, *v;
    float *k_scale, *v_scale;        // e4m3: float32; int4: bf16 (cast where they are used); else unused
};

struct AppendProblem {
    int B, S;                        // sequences; tokens of each, or of all where they are packed
    KvCache cache;
    const void *k, *v;
    int64_t k_stride[3], v_stride[3];  // b, h, s (elements)
    const int32_t *page_table;       // [B, max_pages]
    int max_pages;
    const int32_t *cache_lens, *new_lens;
    const int32_t *starts;           // [B + 1]: where packed sequences begin; null: k, v are [B, H, S, D]
    const double *inv_freq;          // null: no rotation
    int rotary, layout;
    float attention_scale;
};

struct ReadProblem {
    int B, T;                        // sequences, packed tokens
    KvCache cache;
    const int32_t *page_table;
    int max_pages;
    const int32_t *starts;           // [B + 1]
    void *out[2];                    // keys, values
    int64_t out_stride[2][2];        // h, token (elements)
    int wide;                        // the outputs' rows are 32-byte aligned
};

struct CacheAttnProblem {
    int B, Hq, G, Q;                 // query heads, heads per key head, query tokens
    KvCache cache;
    const uint16_t *q;
    int64_t q_stride[3];             // b, h, token (elements)
    const int32_t *page_table;
    int max_pages;
    const int32_t *kv_lens;
    int window, sinks;               // window INT32_MAX: every earlier token
    int causal;                      // 0: rows see every cached token
    int score_kind;
    float score_param, scale;
    uint16_t *out;
    float *lse;
    int *status;                     // device status word
    void *workspace;                 // cache_attention_workspace() bytes
};

cudaError_t launch_rope(const RopeProblem &p, int dtype, cudaStream_t stream);
cudaError_t launch_kv_append(const AppendProblem &p, int src_dtype, int cache_dtype, cudaStream_t stream);
cudaError_t launch_kv_append_packed(const AppendProblem &p, int src_dtype, int cache_dtype, cudaStream_t stream);
cudaError_t launch_kv_append_int4(const AppendProblem &p, int src_dtype, cudaStream_t stream);
cudaError_t launch_kv_read(const ReadProblem &p, int cache_dtype, int out_dtype, cudaStream_t stream);
int64_t cache_attention_workspace(const CacheAttnProblem &p, int cache_dtype);  // bytes
int64_t cache_attention_int4_workspace(const CacheAttnProblem &p);
cudaError_t launch_cache_attention_int4(const CacheAttnProblem &p, cudaStream_t stream);
cudaError_t launch_cache_attention(const CacheAttnProblem &p, int cache_dtype, cudaStream_t stream);

// Angles are kept as turns in 64-bit fixed point: position * frequency wraps
// modulo one turn by itself.  The frequency's turns are within 2^-64 (of
// frequencies up to 2^40), so that the angle of any int32 position is within
// 2^-33 of a turn; the rounded product with a rounded 1 / (2 pi) would be off by
// 2^-25 of a turn at position 2^31 and 0.75 radians per position, and by more
// for larger frequencies.  In float32 the angle of position 131072 would be off
// by 0.004 radians.
//
// In whole numbers: the float64's 53 bits times 128 bits of 1 / (2 pi), shifted.
// Double precision, of which an SM does two operations a clock, took 0.4 us more
// of an appended decoding step's 3.2.
__device__ __forceinline__ uint64_t turns_per_position(double inv_freq) {
    constexpr uint64_t hi = 0x28be60db9391054aull, lo = 0x7f09d5f47d4d3770ull;  // 1 / (2 pi) = (hi 2^64 + lo) 2^-128
    const uint64_t bits = (uint64_t)__double_as_longlong(inv_freq);
    const int exponent = (int)(bits >> 52) & 0x7FF, right = 1075 - exponent;  // |inv_freq| = digits 2^-right
    const uint64_t digits = (bits & 0xFFFFFFFFFFFFFull) | (uint64_t)(exponent != 0) << 52;
    // digits / (2 pi) as top + low 2^-64, and the turns of it that are left modulo one
    const uint64_t part = digits * hi, low = part + __umul64hi(digits, lo), top = __umul64hi(digits, hi) + (low < part);
    uint64_t turns = 0;  // of frequencies below 2^-75, and where a step of the float64 is more than a turn
    if (right > 0 && right < 64) turns = low >> right | top << (64 - right);
    if (right >= 64 && right < 128) turns = top >> (right - 64);
    return inv_freq < 0 ? 0 - turns : turns;
}
// Sine and cosine of a position's angle.  What is left of it beside whole
// quarter turns goes to float32, x in [-1/4, 1/4] half turns: rounding it moves
// the angle by 2^-28 of a turn at most (a rounding of all of it: 2^-26).  There
// the Taylor series of sin(pi x) to x^9 and of cos(pi x) to x^10 leave out less
// than 2^-28 of the result; pi as a sum of two floats keeps the sine's first
// term from losing a bit.  Half the instructions of sincospi, of which a prompt
// appended to a cache needs one per token, pair and run of heads.
__device__ __forceinline__ void sincos_at(uint64_t turns, int32_t position, float *sine, float *cosine) {
    const uint64_t angle = turns * (uint64_t)(int64_t)position;
    const uint32_t quarters = ((uint32_t)(angle >> 32) + 0x20000000u) >> 30;
    const int64_t rest = (int64_t)(angle - ((uint64_t)quarters << 62));
    const float x = (float)(int32_t)(rest >> 30) * 1.1641532182693481e-10f;  // 2^-33
    constexpr double pi = 3.14159265358979323846, p2 = pi * pi;
    constexpr float pi_hi = (float)pi, pi_lo = (float)(pi - (double)(float)pi);
    const float t = x * x;
    float s = fmaf(t, (float)(p2 * p2 * p2 * p2 * pi / 362880), (float)(-p2 * p2 * p2 * pi / 5040));
    s = fmaf(t, s, (float)(p2 * p2 * pi / 120));
    s = fmaf(t, s, (float)(-p2 * pi / 6));
    s = fmaf(t, s, pi_lo);
    s = fmaf(x, pi_hi, x * s);
    float c = fmaf(t, (float)(-p2 * p2 * p2 * p2 * p2 / 3628800), (float)(p2 * p2 * p2 * p2 / 40320));
    c = fmaf(t, c, (float)(-p2 * p2 * p2 / 720));
    c = fmaf(t, c, (float)(p2 * p2 / 24));
    c = fmaf(t, c, (float)(-p2 / 2));
    c = fmaf(t, c, 1.f);
    const float a = quarters & 1u ? c : s, z = quarters & 1u ? s : c;
    *sine = quarters & 2u ? -a : a;
    *cosine = (quarters + 1u) & 2u ? -z : z;
}

}  // namespace flex
