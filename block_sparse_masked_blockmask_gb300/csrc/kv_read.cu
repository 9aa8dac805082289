// Reading a paged cache back: the tokens of packed sequences as contiguous keys
// and values, in bf16 or float32.  Packed token T of sequence b (starts[b] <= T
// < starts[b + 1]) is position T - starts[b]; a position that has no page reads
// as zeros.
//
// Bound by memory, mostly by what it writes (4-bit codes to bf16: 2 bytes
// written for 0.56 read).  A CTA takes a run of tokens: their sequences and pages
// are looked up once into shared memory, then its threads walk (head, token) rows of
// its keys, or of its values.  Measured to bf16: two sequences of 131071 tokens of 8 heads
// of 128 from 4 bits, 238 us or 85% of the copy rate; 24 up to 4095 of 8 heads of 64
// from e4m3, 29 us, 81%.
#include "kv_internal.h"
#include "kv_values.cuh"

namespace flex {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 32;  // of a CTA

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

// N floats (a multiple of 8) to bf16 or float32, in stores of 32 bytes (whole
// sectors: two of 16 cost 20% more time) where the output's rows allow it.
template <int N>
__device__ __forceinline__ void store_values(uint16_t *dst, const float (&x)[N], bool wide) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    if (N >= 16 && wide) {
#pragma unroll
        for (int i = 0; i < N / 2; i += 8) st_global_32B(dst + 2 * i, w + i);
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; i += 4)
            *reinterpret_cast<uint4 *>(dst + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
}
template <int N>
__device__ __forceinline__ void store_values(float *dst, const float (&x)[N], bool wide) {
    if (wide) {
#pragma unroll
        for (int i = 0; i < N; i += 8) st_global_32B(dst + i, reinterpret_cast<const uint32_t *>(x) + i);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(dst + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    }
}

// What a thread reads of a row, and the values that it stands for: N of them,
// from value `first(part)` on.
template <int KIND, int D>
struct Piece;
template <int D>
struct Piece<FLEX_DTYPE_BF16, D> {
    static constexpr int N = 8, P = D / N;
    static __device__ __forceinline__ void read(const KvCache &c, bool, const uint8_t *base, int64_t row, int64_t, int part,
                                                float (&x)[N]) {
        Raw8<uint16_t> raw;
        raw.load(reinterpret_cast<const uint16_t *>(base) + row * D + part * N);
        raw.unpack(x);
    }
};
template <int D>
struct Piece<FLEX_DTYPE_E4M3, D> {
    static constexpr int N = 16, P = D / N;
    static __device__ __forceinline__ void read(const KvCache &c, bool is_v, const uint8_t *base, int64_t row, int64_t page_head,
                                                int part, float (&x)[N]) {
        const uint4 r = *reinterpret_cast<const uint4 *>(base + row * D + part * N);
        const float s = __ldg((is_v ? c.v_scale : c.k_scale) + page_head);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w[i / 2] >> (16 * (i % 2)))));
            float lo, hi;
            asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
                : "=f"(lo), "=f"(hi)
                : "r"(h2));
            x[2 * i] = lo * s;
            x[2 * i + 1] = hi * s;
        }
    }
};
template <int D>
struct Piece<FLEX_DTYPE_INT4, D> {
    // 32 values, those of group `part`: thread p reads the 16 bytes that hold
    // 1024 / D values of every group, and the D / 32 threads of a row swap them
    static constexpr int N = 32, P = D / N;
    static __device__ __forceinline__ void read(const KvCache &c, bool is_v, const uint8_t *base, int64_t row, int64_t, int part,
                                                float (&x)[N]) {
        const uint4 r = *reinterpret_cast<const uint4 *>(base + row * (D / 2) + part * 16);
        const uint16_t *sp = reinterpret_cast<const uint16_t *>(is_v ? c.v_scale : c.k_scale);
        const float s = __uint_as_float((uint32_t)__ldg(is_v ? sp + row : sp + row * P + part) << 16);
        uint32_t w[4];  // of the values in ascending order
        if constexpr (D == 128) {
            // words of group j from thread p: units (2 p, j), (2 p + 1, j)
            uint32_t a[4] = {prmt(r.x, r.z, 0x5410u), prmt(r.x, r.z, 0x7632u), prmt(r.y, r.w, 0x5410u), prmt(r.y, r.w, 0x7632u)};
            // 4 x 4 transpose over the four threads: exchange with the neighbour, then with the one two further on
            const unsigned mask = 0xffffffffu;
            {
                const bool odd = part & 1;
                const uint32_t g0 = __shfl_xor_sync(mask, odd ? a[0] : a[1], 1), g1 = __shfl_xor_sync(mask, odd ? a[2] : a[3], 1);
                if (odd) { a[0] = g0; a[2] = g1; } else { a[1] = g0; a[3] = g1; }
            }
            {
                const bool up = part & 2;
                const uint32_t g0 = __shfl_xor_sync(mask, up ? a[0] : a[2], 2), g1 = __shfl_xor_sync(mask, up ? a[1] : a[3], 2);
                if (up) { a[0] = g0; a[1] = g1; } else { a[2] = g0; a[3] = g1; }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = a[i];
        } else {
            // word i of thread p: units (4 p + i, 0), (4 p + i, 1)
            const uint32_t lo[2] = {prmt(r.x, r.y, 0x5410u), prmt(r.z, r.w, 0x5410u)};  // of group 0
            const uint32_t hi[2] = {prmt(r.x, r.y, 0x7632u), prmt(r.z, r.w, 0x7632u)};  // of group 1
            const bool odd = part & 1;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? lo[i] : hi[i], 1);
                w[i] = odd ? got : lo[i];
                w[2 + i] = odd ? hi[i] : got;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)  // 2^23 + code, less 2^23 + 8: exact
                x[8 * i + e] = (__uint_as_float(((w[i] >> (4 * e)) & 15u) | 0x4B000000u) - 8388616.f) * s;
    }
};

template <int KIND, typename T, int D>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadProblem p) {
    using C = Piece<KIND, D>;
    __shared__ int64_t row_of[kTokens];   // of head 0: page * H * page size + slot; -1: no page; -2: no token
    __shared__ int32_t starts_here[kStartsHere + 1];
    const int token0 = (int)blockIdx.x * kTokens;
    const int32_t *starts = stage_starts(p.starts, p.B, starts_here);
    __syncthreads();
    if (threadIdx.x < kTokens) {
        const int token = token0 + (int)threadIdx.x, b = token < p.T ? sequence_of(starts, p.B, token) : -1;
        int64_t row = -2;
        if (b >= 0) {
            const int64_t position = (int64_t)token - starts[b], entry = position >> p.cache.page_shift;
            const int id = entry < p.max_pages ? __ldg(p.page_table + (int64_t)b * p.max_pages + entry) : -1;
            row = id >= 0 && id < p.cache.num_pages
                      ? (int64_t)id * p.cache.H * p.cache.page + (position & (p.cache.page - 1))
                      : -1;
        }
        row_of[threadIdx.x] = row;
    }
    __syncthreads();
    const bool is_v = blockIdx.z != 0;
    const uint8_t *base = is_v ? p.cache.v : p.cache.k;
    const int part = threadIdx.x % C::P;
    constexpr int kRows = kThreads / C::P;  // rows at a time
    // rows in the order of heads, tokens innermost; all threads of a row walk together
    const int heads = (p.cache.H + (int)gridDim.y - 1) / (int)gridDim.y, h0 = (int)blockIdx.y * heads,
              h1 = min(h0 + heads, p.cache.H);
    for (int i0 = h0 * kTokens; i0 < h1 * kTokens; i0 += kRows) {
        const int i = i0 + (int)threadIdx.x / C::P, h = i / kTokens, tok = i % kTokens;
        const int64_t row0 = h < h1 ? row_of[tok] : -2;
        float x[C::N];
        const bool held = row0 >= 0;
        // a row of the cache in any case (a thread's neighbours swap with it)
        const int64_t row = held ? row0 + (int64_t)h * p.cache.page : 0;
        C::read(p.cache, is_v, base, row, row >> p.cache.page_shift, part, x);
        if (row0 == -2) continue;
        if (!held) {
#pragma unroll
            for (int e = 0; e < C::N; ++e) x[e] = 0.f;
        }
        store_values(static_cast<T *>(p.out[is_v]) + h * p.out_stride[is_v][0] + (int64_t)(token0 + tok) * p.out_stride[is_v][1] +
                         part * C::N,
                     x, p.wide);
    }
}

template <int KIND, typename T>
cudaError_t launch(const ReadProblem &p, cudaStream_t stream) {
    const int64_t tiles = ((int64_t)p.T + kTokens - 1) / kTokens;
    int groups = 1;  // of heads, until there are four CTAs for every SM
    while (groups < p.cache.H && tiles * 2 * groups < 4 * 152) groups *= 2;
    if (groups > p.cache.H) groups = p.cache.H;
    const dim3 grid((unsigned)tiles, (unsigned)groups, 2);
    if (p.cache.D == 64)
        kv_read_kernel<KIND, T, 64><<<grid, kThreads, 0, stream>>>(p);
    else
        kv_read_kernel<KIND, T, 128><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <int KIND>
cudaError_t launch_typed(const ReadProblem &p, int out_dtype, cudaStream_t stream) {
    return out_dtype == FLEX_DTYPE_BF16 ? launch<KIND, uint16_t>(p, stream) : launch<KIND, float>(p, stream);
}

}  // namespace

cudaError_t launch_kv_read(const ReadProblem &p, int cache_dtype, int out_dtype, cudaStream_t stream) {
    if (cache_dtype == FLEX_DTYPE_INT4) return launch_typed<FLEX_DTYPE_INT4>(p, out_dtype, stream);
    if (cache_dtype == FLEX_DTYPE_E4M3) return launch_typed<FLEX_DTYPE_E4M3>(p, out_dtype, stream);
    return launch_typed<FLEX_DTYPE_BF16>(p, out_dtype, stream);
}

}  // namespace flex
