// Attention of a sequence's newest tokens against its paged cache: for every
// query row (token t of Q, head h; position pos = kv_lens[b] - Q + t)
//   s[kv] = score_mod(scale q.k[kv])  for the kv its mask keeps, kv <= pos
//   out   = sum_kv exp(s[kv] - lse) v[kv],   lse = ln sum_kv exp(s[kv])
// in one pass over the keys (running maximum and sum), the query heads that
// share a key head reading it together.
//
// Bound by memory: the visible tokens' keys and values are read once (1 or 2
// bytes a value) for 4 G Q flops per pair of them.  The products run on
// mma.sync m16n8k16: one such tile has 16 keys against 8 query rows, which is
// what a step of decoding has; a tcgen05 tile has 128 rows, and its operands
// would have to pass through shared memory as 16-bit values first, which costs
// more than the product.  At 6.8 TB/s an SM receives 23 e4m3 values a clock; 8
// rows of products on them are 375 flops a clock.
//
//  * Keys go from global memory straight into the A operand of S^T = K Q^T:
//    thread (g, t) of a warp (lane = 4 g + t) loads 16-byte pieces of keys g and
//    g + 8, in a fixed permutation of the head dim that Q's operand follows.
//    Values are the A operand of O^T = V^T P^T: the thread loads the pieces at
//    its own head dims of the tokens 2t, 2t+1, 2t+8, 2t+9 and pairs them with
//    byte permutes.  Neither passes through shared memory.
//  * e4m3 codes convert to fp16 exactly, two per instruction.  Q rows are
//    divided by a power of two first so that they fit fp16 (bf16 values keep
//    all their bits down to 2^-14 of the row's largest).  The page's scale of K
//    multiplies the scores, the one of V the weights: P is kept relative to the
//    largest V scale met, which rescales the accumulators when it grows.
//    A bf16 cache runs the same in bf16.
//  * S^T's accumulators hold keys along lanes' g and rows along t: after
//    exp, one 8 x 8 transpose (movmatrix) per half tile makes them the B
//    operand P^T.  Statistics, sums and accumulators are float32.
//  * The maximum is only raised when a score exceeds it by 2^8 (votes instead of
//    reductions on most steps); weights then stay below 2^8.
//  * A sequence's tokens are split over the warps of a cluster of up to 16 CTAs,
//    tile by tile; the partial results meet in distributed shared memory, so
//    there is no workspace, no second launch and no atomic.
//  * Only tiles at an edge (the last tokens, a window's ends, a bad page)
//    evaluate the mask; there the values of tokens that no row keeps are
//    zeroed, so that whatever lies in those slots has no effect, and where
//    rows of the call differ in what they keep and such a token's value is not
//    finite, the tile's product is done once per query token.
#include <cfloat>
#include <climits>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_internal.h"
#include "ptx.cuh"

namespace flex {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.f;  // raise the running max only beyond 2^8

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
// Two e4m3 codes (low or high half of w) to fp16x2, exactly.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// 8 x 8 transpose of 16-bit values across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Cache data is read once: keep it out of L1.
template <int BYTES>
__device__ __forceinline__ void load_stream(uint32_t *w, const uint8_t *src) {
    if constexpr (BYTES == 8)
        asm volatile("ld.global.nc.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(src));
    else
        asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "l"(src));
}

// D: head dim; E4M3: cache type (else bf16); NT: tiles of 8 query rows.
template <int D, bool E4M3, int NT>
struct Cfg {
    static constexpr int kElem = E4M3 ? 1 : 2;
    static constexpr int kRowBytes = D * kElem;
    // 16-token groups a warp has in flight: 4 KB of keys and 4 KB of values
    static constexpr int kSub = 4096 / (16 * kRowBytes);
    static constexpr int kTokens = 16 * kSub;
    static constexpr int kSteps = D / 16;               // k16 steps of S, m16 tiles of O
    static constexpr int kKWords = kRowBytes / 16;      // words of one key a thread holds
    static constexpr int kVBytes = kRowBytes / 8;       // bytes of one value a thread holds
    static constexpr int kVLoad = kVBytes < 16 ? 8 : 16;
    static constexpr int kRows = 8 * NT;
    static constexpr int kAccStride = D + 4;
    // shared memory: Q operand, then per warp the accumulators and statistics
    static constexpr int kQBytes = NT * kSteps * 32 * 8;
    static constexpr int kAccBytes = kWarps * kRows * kAccStride * 4;
    static constexpr int kSmem = (kQBytes > kAccBytes ? kQBytes : kAccBytes);
};

struct Stats {
    float m[kWarps][32], l[kWarps][32], f[kWarps][32];  // per warp and row
    float cm[32], cl[32];                               // of the CTA
    float qf[32];                                       // the power of two taken off a query row
};

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) cache_attention_kernel(CacheAttnProblem p, int csize,
                                                                                    int row_tiles) {
    using C = Cfg<D, E4M3, NT>;
    constexpr int SUB = C::kSub, KS = C::kSteps;
    namespace cg = cooperative_groups;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Stats st;
    uint2 *qs = reinterpret_cast<uint2 *>(smem);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
    const int rank = (int)(blockIdx.x % csize);
    const int pair = (int)(blockIdx.x / csize);
    const int rt = pair % row_tiles, bh = pair / row_tiles, hk = bh % p.cache.H, b = bh / p.cache.H;
    const int page = p.cache.page;

    // rows of this tile: r = query token * G + head within the group
    const int rows = p.Q * p.G, r0 = rt * C::kRows, r1 = min(r0 + C::kRows, rows) - 1;
    const int tmin = r0 / p.G, tmax = r1 / p.G;
    const int cap = (int)min((int64_t)p.max_pages * page, (int64_t)INT_MAX);
    const int n = min(max(p.kv_lens[b], 0), cap);
    // what any row of the tile keeps: [0, send) and [lo, hi)
    const int hi = p.causal ? max(n - p.Q + tmax + 1, 0) : n;
    const int64_t lo_min = p.causal ? max((int64_t)n - p.Q + tmin - p.window + 1, (int64_t)0) : 0;
    int lo = (int)min(lo_min, (int64_t)hi) / C::kTokens * C::kTokens;
    const int send = min(p.sinks, hi);
    int nsink = (send + C::kTokens - 1) / C::kTokens;
    if (nsink * (int64_t)C::kTokens >= lo) {
        nsink = 0;
        lo = 0;
    }
    const int ntiles = nsink + (hi - lo + C::kTokens - 1) / C::kTokens;
    // what every row keeps, for tiles without mask work
    const int all_hi = p.causal ? n - p.Q + tmin + 1 : (n - p.Q + tmin >= 0 ? n : 0);
    const int64_t all_lo = p.causal ? (int64_t)n - p.Q + tmax - p.window + 1 : 0;
    auto tile_base = [&](int i) { return i < nsink ? i * C::kTokens : lo + (i - nsink) * C::kTokens; };

    const int *table = p.page_table + (int64_t)b * p.max_pages;
    const int64_t page_bytes = (int64_t)page * C::kRowBytes;
    uint32_t kw[SUB][2][C::kKWords], vw[SUB][4][C::kVBytes / 4];
    int64_t ph[SUB], ph_next[SUB];  // page * heads + head of the groups in flight, -1: nothing there
    auto lookup = [&](int base, int64_t (&q)[SUB]) {
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
            const int at = base + 16 * j;
            q[j] = -1;
            if (at < hi && (at + 16 > lo_min || at < send)) {
                const int id = __ldg(table + (at >> p.cache.page_shift));
                if (id >= 0 && id < p.cache.num_pages) q[j] = (int64_t)id * p.cache.H + hk;
            }
        }
    };
    auto load_k = [&](int base, const int64_t (&q)[SUB]) {
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
            const uint8_t *src = p.cache.k + q[j] * page_bytes +
                                 (int64_t)((base + 16 * j) & (page - 1)) * C::kRowBytes + g * C::kRowBytes + t * 16;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int c = 0; c < C::kKWords / 4; ++c) {
                    if (q[j] >= 0)
                        load_stream<16>(&kw[j][r][4 * c], src + r * 8 * C::kRowBytes + c * 64);
                    else
                        kw[j][r][4 * c] = kw[j][r][4 * c + 1] = kw[j][r][4 * c + 2] = kw[j][r][4 * c + 3] = 0u;
                }
        }
    };
    auto load_v = [&](int base, const int64_t (&q)[SUB]) {
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
            const uint8_t *src = p.cache.v + q[j] * page_bytes +
                                 (int64_t)((base + 16 * j) & (page - 1)) * C::kRowBytes + 2 * t * C::kRowBytes +
                                 g * C::kVLoad;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < C::kVBytes / C::kVLoad; ++c) {
                    uint32_t *w = &vw[j][r][c * C::kVLoad / 4];
                    if (q[j] >= 0) {
                        load_stream<C::kVLoad>(w, src + ((r & 1) + (r >> 1) * 8) * C::kRowBytes + c * 128);
                    } else {
#pragma unroll
                        for (int e = 0; e < C::kVLoad / 4; ++e) w[e] = 0u;
                    }
                }
        }
    };

    const int step = csize * kWarps;
    int tile = rank * kWarps + warp;
    if (tile < ntiles) {
        lookup(tile_base(tile), ph);
        load_k(tile_base(tile), ph);
        load_v(tile_base(tile), ph);
    }

    // Q operand: the rows' largest magnitudes first (e4m3), then the fragments
    auto q_row = [&](int r) {
        const int row = r0 + r;
        return p.q + b * p.q_stride[0] + (int64_t)(hk * p.G + row % p.G) * p.q_stride[1] +
               (int64_t)(row / p.G) * p.q_stride[2];
    };
    if constexpr (E4M3) {
        for (int r = warp; r < C::kRows; r += kWarps) {
            uint32_t top = 0u;
            if (r0 + r <= r1) {
                const uint16_t *src = q_row(r);
                for (int d = 4 * lane; d < D; d += 128) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(src + d);
                    top = max(max(w.x & 0x7FFFu, (w.x >> 16) & 0x7FFFu), max(w.y & 0x7FFFu, (w.y >> 16) & 0x7FFFu));
                }
            }
            top = __reduce_max_sync(0xffffffffu, top);
            // exponent field of the largest value; 1 for a row of zeros and
            // for rows with infinities or NaN, whose scores are not finite
            const uint32_t e = top >> 7;
            if (lane == 0) st.qf[r] = e == 0u || e == 255u ? 1.f : __uint_as_float(e << 23);
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < NT * KS * 32; i += kThreads) {
        const int l = i % 32, j = (i / 32) % KS, nt = i / (32 * KS), r = nt * 8 + (l >> 2);
        // the four head dims of step j that lane l's key words hold
        const int d = E4M3 ? (j / 4) * 64 + (l & 3) * 16 + (j % 4) * 4 : (j / 2) * 32 + (l & 3) * 8 + (j % 2) * 4;
        uint2 w = make_uint2(0u, 0u);
        if (r0 + r <= r1) {
            w = *reinterpret_cast<const uint2 *>(q_row(r) + d);
            if constexpr (E4M3) {
                const float f = 1.f / st.qf[r];
                w.x = pack_f16x2(__uint_as_float(w.x << 16) * f, __uint_as_float(w.x & 0xFFFF0000u) * f);
                w.y = pack_f16x2(__uint_as_float(w.y << 16) * f, __uint_as_float(w.y & 0xFFFF0000u) * f);
            }
        }
        qs[i] = w;
    }
    __syncthreads();

    // this thread's rows: columns 2t and 2t + 1 of every row tile
    float slope[NT][2], qscale[NT][2];
    int pos[NT][2], seen[NT][2];  // position, and the last kv it keeps (-1: nothing)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = nt * 8 + 2 * t + u, row = r0 + r;
            const bool live = row <= r1;
            const int h = hk * p.G + (live ? row % p.G : 0);
            pos[nt][u] = n - p.Q + (live ? row / p.G : 0);
            seen[nt][u] = live && pos[nt][u] >= 0 ? (p.causal ? pos[nt][u] : n - 1) : -1;
            qscale[nt][u] = p.scale * (E4M3 ? st.qf[r] : 1.f);
            slope[nt][u] = exp2f(-8.f * (float)(h + 1) / (float)p.Hq);
        }

    float m[NT][2], l[NT][2], acc[NT][KS][4], vref = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -FLT_MAX;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < KS; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
    }

    for (; tile < ntiles; tile += step) {
        const int base = tile_base(tile);
        const bool more = tile + step < ntiles;
        const int next = more ? tile_base(tile + step) : 0;
        if (more) lookup(next, ph_next);
        float ks[SUB], vs[SUB];
        bool whole = base + C::kTokens <= all_hi && (base >= all_lo || base + C::kTokens <= p.sinks);
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
            whole = whole && ph[j] >= 0;
            ks[j] = vs[j] = 1.f;
            if constexpr (E4M3) {
                ks[j] = ph[j] >= 0 ? __ldg(p.cache.k_scale + ph[j]) : 0.f;
                vs[j] = ph[j] >= 0 ? __ldg(p.cache.v_scale + ph[j]) : 0.f;
            }
        }
        // ---- S^T = K Q^T
        float x[NT][SUB][4];
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) x[nt][j][0] = x[nt][j][1] = x[nt][j][2] = x[nt][j][3] = 0.f;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                uint32_t a0, a1, a2, a3;
                if constexpr (E4M3) {
                    a0 = e4m3_lo(kw[j][0][s]);
                    a1 = e4m3_lo(kw[j][1][s]);
                    a2 = e4m3_hi(kw[j][0][s]);
                    a3 = e4m3_hi(kw[j][1][s]);
                } else {
                    a0 = kw[j][0][2 * s];
                    a1 = kw[j][1][2 * s];
                    a2 = kw[j][0][2 * s + 1];
                    a3 = kw[j][1][2 * s + 1];
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint2 q = qs[(nt * KS + s) * 32 + lane];
                    mma16816<E4M3>(x[nt][j], a0, a1, a2, a3, q.x, q.y);
                }
            }
        }
        if (more) load_k(next, ph_next);

        // ---- scores in base-2 units, masked
        float top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            top[nt][0] = top[nt][1] = -INFINITY;
#pragma unroll
            for (int j = 0; j < SUB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int u = e & 1, kv = base + 16 * j + g + (e >> 1) * 8;
                    float s = x[nt][j][e] * (qscale[nt][u] * ks[j]);
                    if (p.score_kind == FLEX_SCORE_SOFTCAP)
                        s = p.score_param * tanhf(s / p.score_param);
                    else if (p.score_kind == FLEX_SCORE_ALIBI)
                        s -= slope[nt][u] * (float)(pos[nt][u] - kv);
                    s *= kLog2e;
                    if (!whole) {
                        const bool keep = ph[j] >= 0 && kv <= seen[nt][u] &&
                                          (pos[nt][u] - kv < p.window || kv < p.sinks);
                        if (!keep) s = -INFINITY;
                    }
                    x[nt][j][e] = s;
                    top[nt][u] = fmaxf(top[nt][u], s);
                }
        }
        // ---- running maximum and V scale
        float vmax = vs[0];
#pragma unroll
        for (int j = 1; j < SUB; ++j) vmax = fmaxf(vmax, vs[j]);
        bool raise = vmax > vref;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) raise |= top[nt][0] > m[nt][0] + kRaise || top[nt][1] > m[nt][1] + kRaise;
        if (__any_sync(0xffffffffu, raise)) {
            const float vnew = fmaxf(vref, vmax), vr = E4M3 ? (vref > 0.f ? vref / vnew : 0.f) : 1.f;
            vref = vnew;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float alpha[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float w = top[nt][u];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, o));
                    const float now = w > m[nt][u] + kRaise ? w : m[nt][u];
                    alpha[u] = exp2f(m[nt][u] - now);
                    m[nt][u] = now;
                    l[nt][u] *= alpha[u];
                    alpha[u] *= vr;
                }
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    acc[nt][i][0] *= alpha[0];
                    acc[nt][i][1] *= alpha[1];
                    acc[nt][i][2] *= alpha[0];
                    acc[nt][i][3] *= alpha[1];
                }
            }
        }
        // ---- values of tokens that no row keeps: zero, whatever lies there
        bool mixed = false;  // a token that some rows keep and some do not has a value that is not finite
        if (!whole) {
#pragma unroll
            for (int j = 0; j < SUB; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int kv = base + 16 * j + 2 * t + (r & 1) + (r >> 1) * 8;
                    const bool any = kv < hi && (kv >= lo_min || kv < send);
                    const bool every = kv < all_hi && (kv >= all_lo || kv < p.sinks);
                    bool odd = false;
#pragma unroll
                    for (int c = 0; c < C::kVBytes / 4; ++c) {
                        if (!any) vw[j][r][c] = 0u;
                        const uint32_t w = vw[j][r][c];
                        if constexpr (E4M3)
                            odd |= __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0u;
                        else
                            odd |= __vcmpgeu2(w & 0x7FFF7FFFu, 0x7F807F80u) != 0u;
                    }
                    mixed |= odd && !every;
                }
            mixed = __any_sync(0xffffffffu, mixed);
        }
        // ---- P, its sum, and P^T as operand
        uint32_t pb[NT][SUB][2];
        float vf[SUB];
#pragma unroll
        for (int j = 0; j < SUB; ++j) vf[j] = E4M3 && vref > 0.f ? vs[j] / vref : 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = ex2_approx(x[nt][j][e] - m[nt][e & 1]);
                    l[nt][e & 1] += w[e];
                }
                if constexpr (E4M3) {
                    pb[nt][j][0] = transpose8(pack_f16x2(w[0] * vf[j], w[1] * vf[j]));
                    pb[nt][j][1] = transpose8(pack_f16x2(w[2] * vf[j], w[3] * vf[j]));
                } else {
                    pb[nt][j][0] = transpose8(pack_bf16x2(w[0], w[1]));
                    pb[nt][j][1] = transpose8(pack_bf16x2(w[2], w[3]));
                }
            }
        // ---- O^T += V^T P^T
        auto product = [&](const uint32_t (&v)[SUB][4][C::kVBytes / 4], const uint32_t (&w)[NT][SUB][2]) {
#pragma unroll
            for (int j = 0; j < SUB; ++j)
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    uint32_t a0, a1, a2, a3;
                    if constexpr (E4M3) {
                        const uint32_t sel = i & 1 ? 0x7362u : 0x5140u;
                        const uint32_t lo2 = prmt(v[j][0][i / 2], v[j][1][i / 2], sel);
                        const uint32_t hi2 = prmt(v[j][2][i / 2], v[j][3][i / 2], sel);
                        a0 = e4m3_lo(lo2);
                        a1 = e4m3_hi(lo2);
                        a2 = e4m3_lo(hi2);
                        a3 = e4m3_hi(hi2);
                    } else {
                        a0 = prmt(v[j][0][i], v[j][1][i], 0x5410u);
                        a1 = prmt(v[j][0][i], v[j][1][i], 0x7632u);
                        a2 = prmt(v[j][2][i], v[j][3][i], 0x5410u);
                        a3 = prmt(v[j][2][i], v[j][3][i], 0x7632u);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816<E4M3>(acc[nt][i], a0, a1, a2, a3, w[nt][j][0], w[nt][j][1]);
                }
        };
        if (!mixed) {
            product(vw, pb);
        } else {
            // one query token's rows at a time, with what they do not keep zeroed
            for (int tok = tmin; tok <= tmax; ++tok) {
                const int at = n - p.Q + tok;
                uint32_t v2[SUB][4][C::kVBytes / 4], p2[NT][SUB][2];
#pragma unroll
                for (int j = 0; j < SUB; ++j) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int kv = base + 16 * j + 2 * t + (r & 1) + (r >> 1) * 8;
                        const bool keep = p.causal ? kv <= at && (at - kv < p.window || kv < p.sinks) : at >= 0 && kv < n;
#pragma unroll
                        for (int c = 0; c < C::kVBytes / 4; ++c) v2[j][r][c] = keep ? vw[j][r][c] : 0u;
                    }
                    // the operand's column is the lane's g
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const bool own = (r0 + nt * 8 + g) / p.G == tok;
                        p2[nt][j][0] = own ? pb[nt][j][0] : 0u;
                        p2[nt][j][1] = own ? pb[nt][j][1] : 0u;
                    }
                }
                // a zero weight of another token's row must not meet a value
                // that is not finite either: those rows' columns keep their sums
                float saved[NT][KS][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < KS; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) saved[nt][i][e] = acc[nt][i][e];
                product(v2, p2);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        if ((r0 + nt * 8 + 2 * t + u) / p.G != tok) {
#pragma unroll
                            for (int i = 0; i < KS; ++i) {
                                acc[nt][i][u] = saved[nt][i][u];
                                acc[nt][i][u + 2] = saved[nt][i][u + 2];
                            }
                        }
            }
        }
        if (more) {
            load_v(next, ph_next);
#pragma unroll
            for (int j = 0; j < SUB; ++j) ph[j] = ph_next[j];
        }
    }

    // ------------------------------------------------- join the warps, the CTAs
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[nt][u] += __shfl_xor_sync(0xffffffffu, l[nt][u], o);
            if (g == 0) {
                st.m[warp][nt * 8 + 2 * t + u] = m[nt][u];
                st.l[warp][nt * 8 + 2 * t + u] = l[nt][u];
            }
        }
    __syncthreads();  // statistics written; Q operand no longer read
    float *accs = reinterpret_cast<float *>(smem);
    if (threadIdx.x < C::kRows) {
        float top = st.m[0][threadIdx.x], sum = 0.f;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, st.m[w][threadIdx.x]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += st.l[w][threadIdx.x] * exp2f(st.m[w][threadIdx.x] - top);
        st.cm[threadIdx.x] = top;
        st.cl[threadIdx.x] = sum;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float f[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = nt * 8 + 2 * t + u;
            float top = st.m[0][r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, st.m[w][r]);
            f[u] = exp2f(m[nt][u] - top) * (E4M3 ? vref : 1.f);
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            // head dims of accumulator rows g and g + 8: neighbours
            const int d = E4M3 ? g * (D / 8) + 2 * i : (i / 4) * 64 + g * 8 + 2 * (i % 4);
            float *at = accs + (warp * C::kRows + nt * 8 + 2 * t) * C::kAccStride + d;
            *reinterpret_cast<float2 *>(at) = make_float2(acc[nt][i][0] * f[0], acc[nt][i][2] * f[0]);
            *reinterpret_cast<float2 *>(at + C::kAccStride) = make_float2(acc[nt][i][1] * f[1], acc[nt][i][3] * f[1]);
        }
    }
    __syncthreads();
    auto store = [&](int r, int d, float a, float z, float top, float sum) {
        const int row = r0 + r, h = hk * p.G + row % p.G, tok = row / p.G;
        const int64_t o = ((int64_t)b * p.Hq + h) * p.Q + tok;
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);  // NaN stays
        *reinterpret_cast<uint32_t *>(p.out + o * D + d) = pack_bf16x2(a * inv, z * inv);
        if (d == 0) p.lse[o] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    };
    const int pairs = (r1 - r0 + 1) * (D / 2);
    for (int i = threadIdx.x; i < pairs; i += kThreads) {
        const int r = i / (D / 2), d = 2 * (i % (D / 2));
        float2 s = *reinterpret_cast<float2 *>(accs + r * C::kAccStride + d);
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float2 o = *reinterpret_cast<float2 *>(accs + (w * C::kRows + r) * C::kAccStride + d);
            s.x += o.x;
            s.y += o.y;
        }
        if (csize == 1)
            store(r, d, s.x, s.y, st.cm[r], st.cl[r]);
        else
            *reinterpret_cast<float2 *>(accs + r * C::kAccStride + d) = s;
    }
    if (csize == 1) return;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();  // every CTA's partial result is in its shared memory
    for (int i = rank * kThreads + threadIdx.x; i < pairs; i += csize * kThreads) {
        const int r = i / (D / 2), d = 2 * (i % (D / 2));
        float top = -FLT_MAX, sum = 0.f, a = 0.f, z = 0.f;
        for (int c = 0; c < csize; ++c) top = fmaxf(top, *cluster.map_shared_rank(&st.cm[r], c));
        for (int c = 0; c < csize; ++c) {
            const float f = exp2f(*cluster.map_shared_rank(&st.cm[r], c) - top);
            const float2 o = *reinterpret_cast<float2 *>(cluster.map_shared_rank(accs + r * C::kAccStride + d, c));
            sum += f * *cluster.map_shared_rank(&st.cl[r], c);
            a += f * o.x;
            z += f * o.y;
        }
        store(r, d, a, z, top, sum);
    }
    cluster.sync();  // no CTA leaves while its shared memory is read
}

template <int D, bool E4M3, int NT>
cudaError_t launch_cache(const CacheAttnProblem &p, cudaStream_t stream) {
    using C = Cfg<D, E4M3, NT>;
    auto kernel = cache_attention_kernel<D, E4M3, NT>;
    const int row_tiles = (p.Q * p.G + C::kRows - 1) / C::kRows;
    const int64_t pairs = (int64_t)p.B * p.cache.H * row_tiles;
    // tokens a row tile may have to read, from what the host knows
    int64_t tokens = (int64_t)p.max_pages * p.cache.page;
    if (p.window != INT_MAX) tokens = tokens < (int64_t)p.window + p.sinks + p.Q ? tokens : (int64_t)p.window + p.sinks + p.Q;
    const int64_t tiles = (tokens + C::kTokens - 1) / C::kTokens;
    // CTAs per sequence and head: enough to fill the GPU, while each warp
    // still has a tile
    int csize = 1;
    while (csize < 16 && pairs * csize < 152 * 6 && (int64_t)csize * kWarps < tiles) csize *= 2;
    if (pairs * csize > INT_MAX) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e == cudaSuccess && csize > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pairs * csize));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)csize;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, csize, row_tiles);
}

template <int D, bool E4M3>
cudaError_t launch_cache_rows(const CacheAttnProblem &p, cudaStream_t stream) {
    const int64_t rows = (int64_t)p.Q * p.G;
    if (rows <= 8) return launch_cache<D, E4M3, 1>(p, stream);
    return launch_cache<D, E4M3, 2>(p, stream);
}

}  // namespace

cudaError_t launch_cache_attention(const CacheAttnProblem &p, int cache_dtype, cudaStream_t stream) {
    if (cache_dtype == FLEX_DTYPE_E4M3)
        return p.cache.D == 64 ? launch_cache_rows<64, true>(p, stream) : launch_cache_rows<128, true>(p, stream);
    return p.cache.D == 64 ? launch_cache_rows<64, false>(p, stream) : launch_cache_rows<128, false>(p, stream);
}

}  // namespace flex
