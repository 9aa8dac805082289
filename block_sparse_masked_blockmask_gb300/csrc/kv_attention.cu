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
// 16 or 8 bytes of shared memory.
template <int BYTES>
__device__ __forceinline__ void load_shared(uint32_t *w, uint32_t addr) {
    if constexpr (BYTES == 8)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    else
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(addr));
}

// D: head dim; E4M3: cache type (else bf16); NT: tiles of 8 query rows.
template <int D, bool E4M3, int NT>
struct Cfg {
    static constexpr int kElem = E4M3 ? 1 : 2;
    static constexpr int kRowBytes = D * kElem;
    static constexpr int kPanelBytes = kRowBytes < 128 ? kRowBytes : 128;  // a row of a staged panel (TMA swizzle span)
    static constexpr int kPanels = kRowBytes / kPanelBytes;
    static constexpr int kTile = 4096;                  // bytes of keys (of values) per step of a warp
    static constexpr int kTokens = kTile / kRowBytes;
    static constexpr int kSub = kTokens / 16;           // groups of 16 tokens per step
    static constexpr int kStages = NT == 1 ? 2 : 3;     // steps in flight per warp
    static constexpr int kSteps = D / 16;               // k16 steps of S, m16 tiles of O
    static constexpr int kKWords = kRowBytes / 16;      // words of one key a thread holds
    static constexpr int kVBytes = kRowBytes / 8;       // bytes of one value a thread holds
    static constexpr int kVLoad = kVBytes < 16 ? 8 : 16;
    static constexpr int kRows = 8 * NT;
    static constexpr int kAccStride = D + 4;
    // shared memory: the warps' rings (over them, at the end, the partial
    // accumulators), then the Q operand
    static constexpr int kRing = kWarps * kStages * 2 * kTile;
    static constexpr int kQBytes = NT * kSteps * 32 * 8;
    static_assert(kWarps * kRows * kAccStride * 4 <= kRing, "partial accumulators fit the rings");
    static constexpr int kSmem = 1024 + kRing + kQBytes;  // 1024: alignment of the swizzle
};

struct Misc {
    uint64_t k_full[kWarps][3], v_full[kWarps][3];
    float m[kWarps][16], l[kWarps][16];  // per warp and row
    float cm[16], cl[16];                // of the CTA
    float qf[16];                        // the power of two taken off a query row
    int abort;
};

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
    cache_attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                           const CacheAttnProblem p, int csize, int row_tiles, int box_rows) {
    using C = Cfg<D, E4M3, NT>;
    constexpr int SUB = C::kSub, KS = C::kSteps, ST = C::kStages;
    namespace cg = cooperative_groups;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Misc ms;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint2 *qs = reinterpret_cast<uint2 *>(smem + C::kRing);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
    const int rank = (int)(blockIdx.x % csize);
    const int pair = (int)(blockIdx.x / csize);
    const int rt = pair % row_tiles, bh = pair / row_tiles, hk = bh % p.cache.H, b = bh / p.cache.H;
    const int page = p.cache.page;
    const int kv_len = __ldg(p.kv_lens + b);
    if (threadIdx.x == 0) {
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
        for (int i = 0; i < kWarps * 3; ++i) {
            mbar_init(&ms.k_full[0][0] + i, 1);
            mbar_init(&ms.v_full[0][0] + i, 1);
        }
        ms.abort = 0;
        fence_barrier_init();
    }

    // rows of this tile: r = query token * G + head within the group
    const int rows = p.Q * p.G, r0 = rt * C::kRows, r1 = min(r0 + C::kRows, rows) - 1;
    const int tmin = r0 / p.G, tmax = r1 / p.G;
    const int n = (int)min((int64_t)max(kv_len, 0), (int64_t)p.max_pages * page);
    // what any row of the tile keeps: [0, send) and [lo_min, hi)
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
    const int step = csize * kWarps;
    int tile = rank * kWarps + warp;
    // Of the 16-token groups of a step: page * heads + head, or -1 where there
    // is nothing that a row keeps, and the page's scales.  The groups of one
    // box share a page.  Lane i holds those of the warp's step 32 k + i, so that
    // the loads' latencies are met once in 32 steps.
    int ph_lane[SUB];
    float ks_lane[SUB], vs_lane[SUB];
    auto lookup = [&](int first) {
        const int mine = first + lane * step;
        const int base = tile_base(mine);
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
            const int at = base + 16 * j, box = at & ~(box_rows - 1);
            ph_lane[j] = -1;
            if (mine < ntiles && box < hi && (box + box_rows > lo_min || box < send)) {
                const int id = __ldg(table + (at >> p.cache.page_shift));
                if (id >= 0 && id < p.cache.num_pages) ph_lane[j] = id * p.cache.H + hk;
            }
            ks_lane[j] = vs_lane[j] = 0.f;
        }
        if constexpr (E4M3) {
#pragma unroll
            for (int j = 0; j < SUB; ++j)
                if (ph_lane[j] >= 0) {
                    ks_lane[j] = __ldg(p.cache.k_scale + ph_lane[j]);
                    vs_lane[j] = __ldg(p.cache.v_scale + ph_lane[j]);
                }
        }
    };
    auto take = [&](int i, int (&ph)[SUB], float (&ks)[SUB], float (&vs)[SUB]) {
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
            ph[j] = __shfl_sync(0xffffffffu, ph_lane[j], i);
            ks[j] = E4M3 ? __shfl_sync(0xffffffffu, ks_lane[j], i) : 1.f;
            vs[j] = E4M3 ? __shfl_sync(0xffffffffu, vs_lane[j], i) : 1.f;
        }
    };
    uint8_t *ring = smem + warp * ST * 2 * C::kTile;
    // one step's keys (or values) into ring slot s (lane 0)
    auto fetch = [&](const CUtensorMap *map, uint8_t *dst, uint64_t *bar, int base, const int (&ph)[SUB]) {
        if (lane == 0) {
            uint32_t bytes = 0;
#pragma unroll
            for (int j = 0; j < SUB; ++j) bytes += ph[j] >= 0 ? 16u * C::kRowBytes : 0u;
            mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
            for (int j = 0; j < SUB; ++j)
                if (ph[j] >= 0 && ((16 * j) & (box_rows - 1)) == 0)
#pragma unroll
                    for (int c = 0; c < C::kPanels; ++c)
                        tma_load_3d(dst + c * C::kTokens * C::kPanelBytes + 16 * j * C::kPanelBytes, map, bar,
                                    c * (C::kPanelBytes / C::kElem), (base + 16 * j) & (page - 1), ph[j]);
        }
    };
    __syncthreads();  // barriers initialised

    // the first steps in flight; ph, ks, vs: of the current step and the ST - 1 behind it
    int ph[ST][SUB];
    float ks[ST][SUB], vs[ST][SUB];
    lookup(tile);
#pragma unroll
    for (int s = 0; s < ST; ++s) {
        take(s, ph[s], ks[s], vs[s]);
        if (tile + s * step < ntiles) {
            const int base = tile_base(tile + s * step);
            uint8_t *slot = ring + s * 2 * C::kTile;
            fetch(&map_k, slot, &ms.k_full[warp][s], base, ph[s]);
            fetch(&map_v, slot + C::kTile, &ms.v_full[warp][s], base, ph[s]);
        }
    }
    int ahead = ST;  // of the warp's steps, the next to be asked for

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
            if (lane == 0) ms.qf[r] = e == 0u || e == 255u ? 1.f : __uint_as_float(e << 23);
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < NT * KS * 32; i += kThreads) {
        const int l = i % 32, j = (i / 32) % KS, nt = i / (32 * KS), r = nt * 8 + (l >> 2), lt = l & 3;
        // the four head dims of step j that lane l's key words hold
        const int d = C::kPanelBytes == 64 ? lt * 16 + j * 4
                      : E4M3               ? (2 * lt + j / 4) * 16 + (j % 4) * 4
                                           : (j / 4) * 64 + (2 * lt + (j % 4) / 2) * 8 + (j % 2) * 4;
        uint2 w = make_uint2(0u, 0u);
        if (r0 + r <= r1) {
            w = *reinterpret_cast<const uint2 *>(q_row(r) + d);
            if constexpr (E4M3) {
                const float f = 1.f / ms.qf[r];
                w.x = pack_f16x2(__uint_as_float(w.x << 16) * f, __uint_as_float(w.x & 0xFFFF0000u) * f);
                w.y = pack_f16x2(__uint_as_float(w.y << 16) * f, __uint_as_float(w.y & 0xFFFF0000u) * f);
            }
        }
        qs[i] = w;
    }
    __syncthreads();
    uint2 qr[NT == 1 ? KS : 1];  // one row tile: the operand stays in registers
    if constexpr (NT == 1) {
#pragma unroll
        for (int s = 0; s < KS; ++s) qr[s] = qs[s * 32 + lane];
    }

    // this thread's rows: columns 2t and 2t + 1 of every row tile
    float slope[NT][2], qscale[NT][2];  // in base-2 units
    int pos[NT][2], seen[NT][2];        // position, and the last kv it keeps (-1: nothing)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = nt * 8 + 2 * t + u, row = r0 + r;
            const bool live = row <= r1;
            const int h = hk * p.G + (live ? row % p.G : 0);
            pos[nt][u] = n - p.Q + (live ? row / p.G : 0);
            seen[nt][u] = live && pos[nt][u] >= 0 ? (p.causal ? pos[nt][u] : n - 1) : -1;
            qscale[nt][u] = p.scale * (E4M3 ? ms.qf[r] : 1.f) * (p.score_kind == FLEX_SCORE_SOFTCAP ? 1.f : kLog2e);
            slope[nt][u] = exp2f(-8.f * (float)(h + 1) / (float)p.Hq) * kLog2e;
        }

    float m[NT][2], l[NT][2], acc[NT][KS][4], vref = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -FLT_MAX;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < KS; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
    }
    // byte offsets of this thread's pieces within a staged tile
    const uint32_t ring_at = smem_u32(ring);
    uint32_t koff[2], voff[2];
    if constexpr (C::kPanelBytes == 128) {
        koff[0] = g * 128 + (((2 * t) ^ g) * 16);
        koff[1] = g * 128 + (((2 * t + 1) ^ g) * 16);
        voff[0] = 2 * t * 128 + ((g ^ (2 * t)) * 16);
        voff[1] = (2 * t + 1) * 128 + ((g ^ (2 * t + 1)) * 16);
    } else {
        koff[0] = koff[1] = g * 64 + ((t ^ (g >> 1)) * 16);
        voff[0] = 2 * t * 64 + (((g >> 1) ^ t) * 16) + (g & 1) * 8;
        voff[1] = voff[0] + 64;
    }

    int slot = 0;
    uint32_t phase = 0;
    bool ok = true, refetched = false;  // refetched: this slot's next keys were already asked for
    for (; tile < ntiles; tile += step) {
        const int base = tile_base(tile);
        const bool more = tile + ST * step < ntiles;
        const int next = more ? tile_base(tile + ST * step) : 0;
        int ph_next[SUB];
        float ks_next[SUB], vs_next[SUB];
        if (more && ahead % 32 == 0) lookup(tile + ST * step);
        take(ahead % 32, ph_next, ks_next, vs_next);
        ++ahead;
        bool whole = base + C::kTokens <= all_hi && (base >= all_lo || base + C::kTokens <= p.sinks);
#pragma unroll
        for (int j = 0; j < SUB; ++j) whole = whole && ph[0][j] >= 0;
        const uint32_t k_at = ring_at + slot * 2 * C::kTile, v_at = k_at + C::kTile;
        // ---- S^T = K Q^T
        if (!__all_sync(0xffffffffu, mbar_wait(&ms.k_full[warp][slot], phase, &ms.abort))) {
            ok = false;
            break;
        }
        float x[NT][SUB][4];
        uint32_t kw[SUB][2][C::kKWords];
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) x[nt][j][0] = x[nt][j][1] = x[nt][j][2] = x[nt][j][3] = 0.f;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int c = 0; c < C::kKWords / 4; ++c)
                    load_shared<16>(&kw[j][r][4 * c], k_at + koff[c & 1] + (c >> 1) * C::kTokens * C::kPanelBytes +
                                                          (16 * j + 8 * r) * C::kPanelBytes);
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
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
                    const uint2 q = NT == 1 ? qr[NT == 1 ? s : 0] : qs[(nt * KS + s) * 32 + lane];
                    mma16816<E4M3>(x[nt][j], a0, a1, a2, a3, q.x, q.y);
                }
            }
        __syncwarp();  // every lane has read the keys
        if (more) fetch(&map_k, ring + slot * 2 * C::kTile, &ms.k_full[warp][slot], next, ph_next);

        // ---- scores in base-2 units, masked
        float top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < SUB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[nt][j][e] *= qscale[nt][e & 1] * ks[0][j];
        if (p.score_kind == FLEX_SCORE_SOFTCAP) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < SUB; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[nt][j][e] = p.score_param * tanhf(x[nt][j][e] / p.score_param) * kLog2e;
        } else if (p.score_kind == FLEX_SCORE_ALIBI) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < SUB; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[nt][j][e] -= slope[nt][e & 1] * (float)(pos[nt][e & 1] - (base + 16 * j + g + (e >> 1) * 8));
        }
        if (!whole) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < SUB; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int u = e & 1, kv = base + 16 * j + g + (e >> 1) * 8;
                        const bool keep = ph[0][j] >= 0 && kv <= seen[nt][u] &&
                                          (pos[nt][u] - kv < p.window || kv < p.sinks);
                        if (!keep) x[nt][j][e] = -INFINITY;
                    }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            top[nt][0] = fmaxf(x[nt][0][0], x[nt][0][2]);
            top[nt][1] = fmaxf(x[nt][0][1], x[nt][0][3]);
#pragma unroll
            for (int j = 1; j < SUB; ++j) {
                top[nt][0] = fmax3(top[nt][0], x[nt][j][0], x[nt][j][2]);
                top[nt][1] = fmax3(top[nt][1], x[nt][j][1], x[nt][j][3]);
            }
        }
        // ---- running maximum and V scale
        float vmax = vs[0][0];
#pragma unroll
        for (int j = 1; j < SUB; ++j) vmax = fmaxf(vmax, vs[0][j]);
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
        // ---- P, its sum, and P^T as operand
        uint32_t pb[NT][SUB][2];
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
            const float vf = !E4M3 || vs[0][j] == vref ? 1.f : vs[0][j] / vref;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = ex2_approx(x[nt][j][e] - m[nt][e & 1]);
                    l[nt][e & 1] += w[e];
                }
                if constexpr (E4M3) {
                    pb[nt][j][0] = transpose8(pack_f16x2(w[0] * vf, w[1] * vf));
                    pb[nt][j][1] = transpose8(pack_f16x2(w[2] * vf, w[3] * vf));
                } else {
                    pb[nt][j][0] = transpose8(pack_bf16x2(w[0], w[1]));
                    pb[nt][j][1] = transpose8(pack_bf16x2(w[2], w[3]));
                }
            }
        }
        // ---- O^T += V^T P^T
        if (!__all_sync(0xffffffffu, mbar_wait(&ms.v_full[warp][slot], phase, &ms.abort))) {
            ok = false;
            refetched = more;
            break;
        }
        auto load_v = [&](int j, uint32_t (&v)[4][C::kVBytes / 4]) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < C::kVBytes / C::kVLoad; ++c)
                    load_shared<C::kVLoad>(&v[r][c * 4], v_at + voff[r & 1] + c * C::kTokens * C::kPanelBytes +
                                                             (16 * j + 8 * (r >> 1)) * C::kPanelBytes);
        };
        auto product = [&](const uint32_t (&v)[4][C::kVBytes / 4], int j, auto &&weight) {
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                uint32_t a0, a1, a2, a3;
                if constexpr (E4M3) {
                    const uint32_t sel = i & 1 ? 0x7362u : 0x5140u;
                    const uint32_t lo2 = prmt(v[0][i / 2], v[1][i / 2], sel);
                    const uint32_t hi2 = prmt(v[2][i / 2], v[3][i / 2], sel);
                    a0 = e4m3_lo(lo2);
                    a1 = e4m3_hi(lo2);
                    a2 = e4m3_lo(hi2);
                    a3 = e4m3_hi(hi2);
                } else {
                    a0 = prmt(v[0][i], v[1][i], 0x5410u);
                    a1 = prmt(v[0][i], v[1][i], 0x7632u);
                    a2 = prmt(v[2][i], v[3][i], 0x5410u);
                    a3 = prmt(v[2][i], v[3][i], 0x7632u);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16816<E4M3>(acc[nt][i], a0, a1, a2, a3, weight(nt, 0), weight(nt, 1));
            }
        };
        if (whole) {
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                uint32_t v[4][C::kVBytes / 4];
                load_v(j, v);
                product(v, j, [&](int nt, int e) { return pb[nt][j][e]; });
            }
        } else {
            // values of tokens that no row keeps: zero, whatever lies there
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                uint32_t v[4][C::kVBytes / 4];
                load_v(j, v);
                bool mixed = false;  // a token that some rows keep and some do not has a value that is not finite
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int kv = base + 16 * j + 2 * t + (r & 1) + (r >> 1) * 8;
                    const bool any = ph[0][j] >= 0 && kv < hi && (kv >= lo_min || kv < send);
                    const bool every = kv < all_hi && (kv >= all_lo || kv < p.sinks);
                    bool odd = false;
#pragma unroll
                    for (int c = 0; c < C::kVBytes / 4; ++c) {
                        if (!any) v[r][c] = 0u;
                        if constexpr (E4M3)
                            odd |= __vcmpeq4(v[r][c] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0u;
                        else
                            odd |= __vcmpgeu2(v[r][c] & 0x7FFF7FFFu, 0x7F807F80u) != 0u;
                    }
                    mixed |= odd && !every;
                }
                if (!__any_sync(0xffffffffu, mixed)) {
                    product(v, j, [&](int nt, int e) { return pb[nt][j][e]; });
                    continue;
                }
                // one query token's rows at a time, with what they do not keep
                // zeroed; the other rows' columns keep their sums, since their
                // zero weights must not meet a value that is not finite either
#pragma unroll 1
                for (int tok = tmin; tok <= tmax; ++tok) {
                    const int at = n - p.Q + tok;
                    float saved[NT][KS][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < KS; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) saved[nt][i][e] = acc[nt][i][e];
                    load_v(j, v);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int kv = base + 16 * j + 2 * t + (r & 1) + (r >> 1) * 8;
                        const bool keep =
                            p.causal ? kv <= at && (at - kv < p.window || kv < p.sinks) : at >= 0 && kv < n;
#pragma unroll
                        for (int c = 0; c < C::kVBytes / 4; ++c) v[r][c] = keep ? v[r][c] : 0u;
                    }
                    product(v, j, [&](int nt, int e) {  // the operand's column is the lane's g
                        return (r0 + nt * 8 + g) / p.G == tok ? pb[nt][j][e] : 0u;
                    });
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
        }
        __syncwarp();  // every lane has read the values
        if (more) fetch(&map_v, ring + slot * 2 * C::kTile + C::kTile, &ms.v_full[warp][slot], next, ph_next);
#pragma unroll
        for (int s = 0; s + 1 < ST; ++s)
#pragma unroll
            for (int j = 0; j < SUB; ++j) ph[s][j] = ph[s + 1][j], ks[s][j] = ks[s + 1][j], vs[s][j] = vs[s + 1][j];
#pragma unroll
        for (int j = 0; j < SUB; ++j) ph[ST - 1][j] = ph_next[j], ks[ST - 1][j] = ks_next[j], vs[ST - 1][j] = vs_next[j];
        if (++slot == ST) {
            slot = 0;
            phase ^= 1u;
        }
    }
    if (!ok) {
        // a copy did not arrive in time: report it, and give the copies still
        // under way (this slot's and the later ones') the same time again
        // before shared memory is used for anything else
        ms.abort = 1;
        if (lane == 0) atomicExch(p.status, kDeviceTimeout);
        volatile int keep_waiting = 0;
        for (int s = 0; s < ST; ++s) {
            const int at = (slot + s) % ST;
            const uint32_t par = phase ^ (slot + s >= ST ? 1u : 0u);
            if (tile + s * step >= ntiles) break;
            mbar_wait(&ms.k_full[warp][at], par, &keep_waiting);
            mbar_wait(&ms.v_full[warp][at], par, &keep_waiting);
        }
        if (refetched) mbar_wait(&ms.k_full[warp][slot], phase ^ 1u, &keep_waiting);
    }

    // ------------------------------------------------- join the warps, the CTAs
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[nt][u] += __shfl_xor_sync(0xffffffffu, l[nt][u], o);
            if (g == 0) {
                ms.m[warp][nt * 8 + 2 * t + u] = m[nt][u];
                ms.l[warp][nt * 8 + 2 * t + u] = l[nt][u];
            }
        }
    __syncthreads();  // statistics written; the rings and the Q operand no longer read
    float *accs = reinterpret_cast<float *>(smem);
    if (threadIdx.x < C::kRows) {
        float top = ms.m[0][threadIdx.x], sum = 0.f;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, ms.m[w][threadIdx.x]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += ms.l[w][threadIdx.x] * exp2f(ms.m[w][threadIdx.x] - top);
        ms.cm[threadIdx.x] = top;
        ms.cl[threadIdx.x] = sum;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float f[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = nt * 8 + 2 * t + u;
            float top = ms.m[0][r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) top = fmaxf(top, ms.m[w][r]);
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
            store(r, d, s.x, s.y, ms.cm[r], ms.cl[r]);
        else
            *reinterpret_cast<float2 *>(accs + r * C::kAccStride + d) = s;
    }
    if (csize == 1) return;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();  // every CTA's partial result is in its shared memory
    for (int i = rank * kThreads + threadIdx.x; i < pairs; i += csize * kThreads) {
        const int r = i / (D / 2), d = 2 * (i % (D / 2));
        float top = -FLT_MAX, sum = 0.f, a = 0.f, z = 0.f;
        for (int c = 0; c < csize; ++c) top = fmaxf(top, *cluster.map_shared_rank(&ms.cm[r], c));
        for (int c = 0; c < csize; ++c) {
            const float f = exp2f(*cluster.map_shared_rank(&ms.cm[r], c) - top);
            const float2 o = *reinterpret_cast<float2 *>(cluster.map_shared_rank(accs + r * C::kAccStride + d, c));
            sum += f * *cluster.map_shared_rank(&ms.cl[r], c);
            a += f * o.x;
            z += f * o.y;
        }
        store(r, d, a, z, top, sum);
    }
    cluster.sync();  // no CTA leaves while its shared memory is read
}

// The cache's keys or values as [pages * heads][page][D]: boxes of box_rows
// tokens by one panel.
template <int D, bool E4M3>
bool make_cache_map(CUtensorMap *map, const void *base, const KvCache &c, int box_rows) {
    using C = Cfg<D, E4M3, 1>;
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)c.page, (uint64_t)c.num_pages * c.H};
    const uint64_t strides[2] = {(uint64_t)C::kRowBytes, (uint64_t)C::kRowBytes * c.page};
    const uint32_t box[3] = {(uint32_t)(C::kPanelBytes / C::kElem), (uint32_t)box_rows, 1};
    return make_tile_map_3d(map, base, E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims,
                            strides, box,
                            C::kPanelBytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
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
    const int box_rows = p.cache.page < C::kTokens ? p.cache.page : C::kTokens;
    CUtensorMap map_k, map_v;
    if (!make_cache_map<D, E4M3>(&map_k, p.cache.k, p.cache, box_rows) ||
        !make_cache_map<D, E4M3>(&map_v, p.cache.v, p.cache, box_rows))
        return cudaErrorInvalidValue;
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
    return cudaLaunchKernelEx(&cfg, kernel, map_k, map_v, p, csize, row_tiles, box_rows);
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
