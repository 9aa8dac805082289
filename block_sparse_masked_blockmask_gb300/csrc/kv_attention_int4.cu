// Attention of a sequence's newest tokens against a paged cache of 4-bit codes:
// what kv_attention.cu computes, with
//   k[d] = (code - 8) ks[token][d / 32],   v[d] = (code - 8) vs[token].
//
// Bound by memory: D + D / 16 + 2 bytes of a visible token and head are read once
// for 4 G Q D flops.  At the copy rate an SM receives 45 codes a clock, so what
// binds beside the memory is the work on them: a code costs a quarter to a third
// of an instruction of a warp's lane to become a 16-bit number, the same again
// for its part of scales, pairing and products.
//
// The list of steps, the rings, the tiles of m16n8k16 products and the join are
// those of kv_attention.cu.  What differs:
//  * The order of codes in a row gives every lane what it multiplies.  Keys: lane
//    (g, t) reads piece t of keys g and g + 8, eight values of each group of 32
//    (all groups), and one byte permute per group puts them in one word: two
//    k16 steps of that group.  Values: it reads piece g of its four tokens, four
//    values of every group, and a byte permute pairs two tokens' 16-bit units.
//    Then the code at nibble n of both halves of a word is one operand register.
//  * Codes become fp16 exactly: or-ed into the mantissa of 1024 (code + 1024, or
//    16 code + 1024 for the upper nibble of a byte), less its offset.
//  * A key's products are summed in float32 group by group and then scaled, two
//    keys a lane: 4 multiply-adds for 512 codes, where scaling the codes would
//    take 8 and round them.
//  * The scale of a value is put on the weights, p = exp2(x - m) vs, which are then
//    rounded to fp16 (11 bits).  m is not the running maximum of the scores x but
//    that of x + log2 vs, so that whatever the scales are, the largest p of a row
//    is between 2^7 and 2^15 and fp16's smallest step 2^-31 of it: a token of small
//    values keeps its bits exactly where it matters to the row.  The sum of
//    weights is taken relative to the same m, before vs.  Scales below 2^-60 count as
//    2^-60 in m, so that weights without their scale stay below 2^75.
#include "kv_attention_common.cuh"

namespace flex {
namespace {

constexpr float kLeastRef = 0x1p-60f;

// fp16x2 of the codes at nibble N of both halves of a word, less 8, exactly.
template <int N>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w) {
    const uint32_t x = N >= 2 ? w >> 8 : w;
    uint32_t r;
    if constexpr (N % 2 == 0)
        asm("{\n\t.reg .b32 h;\n\tlop3.b32 h, %1, 0x000F000F, 0x64006400, 0xEA;\n\t"
            "add.rn.f16x2 %0, h, %2;\n\t}" : "=r"(r) : "r"(x), "r"(0xE408E408u));  // - 1032
    else
        asm("{\n\t.reg .b32 h;\n\tlop3.b32 h, %1, 0x00F000F0, 0x64006400, 0xEA;\n\t"
            "fma.rn.f16x2 %0, h, %2, %3;\n\t}" : "=r"(r) : "r"(x), "r"(0x2C002C00u), "r"(0xD480D480u));  // / 16, - 72
    return r;
}

template <int D, int NT>
struct Cfg4 {
    static constexpr int kRowBytes = D / 2;             // of codes; TMA swizzle span
    static constexpr int kGroups = D / 32;
    static constexpr int kTokens = 64;                  // of a step
    static constexpr int kSub = kTokens / 16;
    static constexpr int kStages = 2;
    static constexpr int kSteps = D / 16;               // k16 steps of S, m16 tiles of O
    static constexpr int kRows = 8 * NT;
    static constexpr int kCodes = kTokens * kRowBytes;  // bytes of a step's keys, or values
    static constexpr int kKeyScales = kTokens * kGroups * 2, kValueScales = kTokens * 2;
    static constexpr int kSlot = (2 * kCodes + kKeyScales + kValueScales + 511) / 512 * 512;
    static constexpr int kRing = kStages * kSlot;
    static constexpr int kQBytes = NT * kSteps * 32 * 8;
    static constexpr int kSmem = 1024 + kWarps * (kRing + kQBytes);
};

struct Misc4 {
    uint64_t k_full[kWarps][2], v_full[kWarps][2];
    int64_t sums[kWarps];
    int abort;
};

template <int D, int NT, bool CAP>
__global__ void __launch_bounds__(kThreads, 2)
    cache_attention_int4_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                                const CacheAttnProblem p, int row_tiles, int box_rows) {
    using C = Cfg4<D, NT>;
    constexpr int SUB = C::kSub, KS = C::kSteps, ST = C::kStages, J = C::kGroups;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Misc4 ms;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem + warp * C::kRing;
    const int page = p.cache.page;
    // the joining launch may start while this one runs: it waits for its end
    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x == 0) {
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_v);
        for (int w = 0; w < kWarps; ++w)
            for (int s = 0; s < ST; ++s) {
                mbar_init(&ms.k_full[w][s], 1);
                mbar_init(&ms.v_full[w][s], 1);
            }
        ms.abort = 0;
        fence_barrier_init();
    }
    // ---- the warp's share of the list
    const int pairs_per_seq = p.cache.H * row_tiles;  // (head, row tile) pairs, the row tiles innermost
    int b, worker, steps;
    int64_t off;
    if (!take_share<C::kTokens>(p, pairs_per_seq, ms.sums, b, off, steps, worker)) return;

    // ---- steps ahead of the computation.  Lane i looks up the warp's step
    // 32 k + i: its first token, and of its 16-token groups page * heads + head,
    // or -1 where there is nothing that a row keeps.  The groups of one box share
    // a page.
    int look_b = b;
    int64_t look_off = off;
    int looked = 0;
    int base_lane = 0, ph_lane[SUB];
    auto lookup = [&]() {
        int lb = look_b;
        int64_t lo_ = look_off + lane;
        Steps sq = steps_of<C::kTokens>(p, __ldg(p.kv_lens + lb));
        while (lo_ >= (int64_t)sq.count * pairs_per_seq && lb + 1 < p.B) {
            lo_ -= (int64_t)sq.count * pairs_per_seq;
            sq = steps_of<C::kTokens>(p, __ldg(p.kv_lens + ++lb));
        }
        const bool live = looked + lane < steps;
        const int pair = (int)(lo_ / sq.count), hk = pair / row_tiles, r0 = pair % row_tiles * C::kRows;
        const int tmin = r0 / p.G, tmax = (min(r0 + C::kRows, p.Q * p.G) - 1) / p.G;
        const int hi = p.causal ? max(sq.n - p.Q + tmax + 1, 0) : sq.n;
        const int64_t lo_min = p.causal ? max((int64_t)sq.n - p.Q + tmin - p.window + 1, (int64_t)0) : 0;
        const int send = min(p.sinks, hi);
        base_lane = sq.base((int)(lo_ % sq.count), C::kTokens);
        const int *table = p.page_table + (int64_t)lb * p.max_pages;
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
            const int at = base_lane + 16 * j, box = at & ~(box_rows - 1);
            ph_lane[j] = -1;
            if (live && box < hi && (box + box_rows > lo_min || box < send)) {
                const int id = __ldg(table + (at >> p.cache.page_shift));
                if (id >= 0 && id < p.cache.num_pages) ph_lane[j] = id * p.cache.H + hk;
            }
        }
        // the next batch begins where lane 31's successor would be
        look_b = __shfl_sync(0xffffffffu, lb, 31);
        look_off = __shfl_sync(0xffffffffu, lo_, 31) + 1;
        looked += 32;
    };
    // one step's keys (or values) and their scales into ring slot `slot` (lane 0); `after` is 0
    auto fetch = [&](bool is_v, int slot, uint32_t after, int base, const int (&ph)[SUB]) {
        if (lane == 0) {
            uint8_t *codes = ring + slot * C::kSlot + (is_v ? C::kCodes : 0) + after;
            uint8_t *scales = ring + slot * C::kSlot + 2 * C::kCodes + (is_v ? C::kKeyScales : 0) + after;
            uint64_t *bar = is_v ? &ms.v_full[warp][slot] : &ms.k_full[warp][slot];
            const int row = is_v ? 2 : 2 * J;  // bytes of a token's scales
            const uint8_t *from = reinterpret_cast<const uint8_t *>(is_v ? p.cache.v_scale : p.cache.k_scale);
            uint32_t bytes = 0;
#pragma unroll
            for (int j = 0; j < SUB; ++j) bytes += ph[j] >= 0 ? 16u * (C::kRowBytes + row) : 0u;
            mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
            for (int j = 0; j < SUB; ++j)
                if (ph[j] >= 0 && ((16 * j) & (box_rows - 1)) == 0) {
                    const int at = (base + 16 * j) & (page - 1);
                    tma_load_3d(codes + 16 * j * C::kRowBytes, is_v ? &map_v : &map_k, bar, 0, at, ph[j]);
                    bulk_load(scales + 16 * j * row, from + ((int64_t)ph[j] * page + at) * row, box_rows * row, bar);
                }
        }
    };
    // of the current step and the ST - 1 behind it
    int base_of[ST], ph[ST][SUB];
    auto take_place = [&](int i, int &base, int (&to)[SUB]) {
        base = __shfl_sync(0xffffffffu, base_lane, i);
#pragma unroll
        for (int j = 0; j < SUB; ++j) to[j] = __shfl_sync(0xffffffffu, ph_lane[j], i);
    };
    lookup();
#pragma unroll
    for (int s = 0; s < ST; ++s) {
        take_place(s, base_of[s], ph[s]);
        if (s < steps) {
            fetch(false, s, 0u, base_of[s], ph[s]);
            fetch(true, s, 0u, base_of[s], ph[s]);
        }
    }

    const uint32_t nothing = (uint32_t)p.cache.page & 1u;  // 0, which the compiler does not know
    // byte offsets of this lane's pieces within a staged tile (TMA swizzle of the row's span)
    const uint32_t ring_at = smem_u32(ring);
    uint32_t koff, voff;
    if constexpr (D == 128) {
        koff = g * 64 + ((t ^ (g >> 1)) * 16);
        voff = 2 * t * 64 + (((g >> 1) ^ t) * 16) + (g & 1) * 8;
    } else {
        koff = g * 32 + (((t >> 1) ^ (g >> 2)) * 16) + (t & 1) * 8;
        voff = 2 * t * 32 + (((g >> 2) ^ (t >> 1)) * 16) + (g & 3) * 4;
    }

    // ---- the pair being computed
    Steps sq = steps_of<C::kTokens>(p, __ldg(p.kv_lens + b));
    int pair = (int)(off / sq.count), at_step = (int)(off % sq.count);
    bool entering = true, whole_start = false;
    int hk = 0, r0 = 0, r1 = 0, n = 0;
    int all_hi = 0, all_lo = 0;
    float slope[NT][2], qscale[NT][2];  // of this thread's rows, columns 2t and 2t + 1 of each row tile (base-2 units)
    int pos[NT][2], seen[NT][2];        // position, and the last kv it keeps (-1: nothing)
    float m[NT][2], l[NT][2], acc[NT][KS][4];
    uint2 *qs = reinterpret_cast<uint2 *>(smem + kWarps * C::kRing + warp * C::kQBytes);

    // ---- the end of a piece: the pair's rows where the warp covered all of its
    // steps, else a partial result
    auto finish = [&](bool whole_end) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[nt][u] += __shfl_xor_sync(0xffffffffu, l[nt][u], o);
        float *part = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(p.workspace) + workspace_partials(p.B)) +
                      (2 * (int64_t)worker + whole_start) * partial_floats(C::kRows, D);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = nt * 8 + 2 * t + u;
                if (r0 + r > r1) continue;
                // head dims of accumulator rows g and g + 8 of tile i: neighbours
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    const int d = 32 * (i / 2) + 4 * g + 2 * (i % 2);
                    if (whole_start && whole_end)
                        store_pair<D>(p, b, hk, r0 + r, d, acc[nt][i][u], acc[nt][i][u + 2], m[nt][u], l[nt][u]);
                    else
                        *reinterpret_cast<float2 *>(part + r * D + d) = make_float2(acc[nt][i][u], acc[nt][i][u + 2]);
                }
                if (!(whole_start && whole_end) && g == 0)
                    *reinterpret_cast<float2 *>(part + C::kRows * D + 2 * r) = make_float2(m[nt][u], l[nt][u]);
            }
    };

    int slot = 0;
    uint32_t phase = 0;
    bool ok = true, refetched = false;  // refetched: this slot's next keys were already asked for
    int it = 0;
    for (; it < steps; ++it) {
        if (entering) {
            entering = false;
            whole_start = at_step == 0;
            n = sq.n;
            hk = pair / row_tiles;
            // rows of this tile: r = query token * G + head within the group
            r0 = pair % row_tiles * C::kRows;
            r1 = min(r0 + C::kRows, p.Q * p.G) - 1;
            const int tmin = r0 / p.G, tmax = r1 / p.G;
            // what every row keeps, for steps without mask work
            all_hi = p.causal ? n - p.Q + tmin + 1 : (n - p.Q + tmin >= 0 ? n : 0);
            all_lo = p.causal ? (int)max((int64_t)n - p.Q + tmax - p.window + 1, (int64_t)0) : 0;
            // Q operand: lane (g, t) takes row g at the head dims of its key pieces
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = r0 + nt * 8 + g;
                const bool live = row <= r1;
                const uint16_t *src = p.q + b * p.q_stride[0] +
                                      (int64_t)(hk * p.G + (live ? row % p.G : 0)) * p.q_stride[1] +
                                      (int64_t)(live ? row / p.G : 0) * p.q_stride[2];
                uint4 w[J];
                uint32_t top = 0u;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    w[j] = live ? *reinterpret_cast<const uint4 *>(src + 32 * j + 8 * t) : make_uint4(0, 0, 0, 0);
                    const uint32_t x[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, max(x[e] & 0x7FFFu, (x[e] >> 16) & 0x7FFFu));
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // rows are divided by the power of two of their largest magnitude, so
                // that they fit fp16 (bf16 values keep all their bits down to 2^-14
                // of it); by 1 where they are zero or not finite
                const uint32_t e = top >> 7;
                const float qf = e == 0u || e == 255u ? 1.f : __uint_as_float(e << 23), f = 1.f / qf;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    // values 0 .. 7 as the pairs (0, 4), (1, 5), (2, 6), (3, 7)
                    const uint32_t lo[2] = {w[j].x, w[j].y}, hi[2] = {w[j].z, w[j].w};
                    uint32_t r[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t a = lo[c / 2], z = hi[c / 2];
                        r[c] = pack_f16x2(__uint_as_float(c % 2 ? a & 0xFFFF0000u : a << 16) * f,
                                          __uint_as_float(c % 2 ? z & 0xFFFF0000u : z << 16) * f);
                    }
                    // read back by this lane alone
                    qs[(nt * KS + 2 * j) * 32 + lane] = make_uint2(r[0], r[1]);
                    qs[(nt * KS + 2 * j + 1) * 32 + lane] = make_uint2(r[2], r[3]);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int rw = r0 + nt * 8 + 2 * t + u;
                    const bool in = rw <= r1;
                    pos[nt][u] = n - p.Q + (in ? rw / p.G : 0);
                    seen[nt][u] = in && pos[nt][u] >= 0 ? (p.causal ? pos[nt][u] : n - 1) : -1;
                    qscale[nt][u] = p.scale * __shfl_sync(0xffffffffu, qf, (2 * t + u) * 4) * (CAP ? 1.f : kLog2e);
                    slope[nt][u] = exp2f(-8.f * (float)(hk * p.G + (in ? rw % p.G : 0) + 1) / (float)p.Hq) * kLog2e;
                    m[nt][u] = -FLT_MAX;
                    l[nt][u] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < KS; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
            }
        }
        const int base = base_of[0];
        const bool more = it + ST < steps;
        int base_next, ph_next[SUB];
        if (more && it + ST == looked) lookup();
        take_place((it + ST) % 32, base_next, ph_next);
        bool whole = base + C::kTokens <= all_hi && (base >= all_lo || base + C::kTokens <= p.sinks);
#pragma unroll
        for (int j = 0; j < SUB; ++j) whole = whole && ph[0][j] >= 0;
        const uint32_t k_at = ring_at + slot * C::kSlot, v_at = k_at + C::kCodes, ks_at = k_at + 2 * C::kCodes,
                       vs_at = ks_at + C::kKeyScales;
        // ---- S^T = K Q^T
        if (!__all_sync(0xffffffffu, mbar_wait(&ms.k_full[warp][slot], phase, &ms.abort))) {
            ok = false;
            break;
        }
        uint32_t kw[SUB][2][J], kscale[SUB][2][J / 2];
#pragma unroll
        for (int j = 0; j < SUB; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                load_shared<4 * J>(kw[j][r], k_at + koff + (16 * j + 8 * r) * C::kRowBytes);
                load_words<J / 2>(kscale[j][r], ks_at + (16 * j + 8 * r + g) * 2 * J);
            }
        __syncwarp();
        if (more)  // the slot is free as soon as its words are in registers
            fetch(false, slot, zero_after(kscale[SUB - 1][1][J / 2 - 1] ^ kw[SUB - 1][1][J - 1], nothing),
                  base_next, ph_next);
        float x[NT][SUB][4];
#pragma unroll
        for (int i = 0; i < J; ++i) {
            uint2 q[2][NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                q[0][nt] = qs[(nt * KS + 2 * i) * 32 + lane];
                q[1][nt] = qs[(nt * KS + 2 * i + 1) * 32 + lane];
            }
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                uint32_t w[2];  // the group's eight codes of keys g and g + 8
                float s[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t sel = i % 2 ? 0x7632u : 0x5410u;
                    w[r] = prmt(kw[j][r][i / 2], kw[j][r][J / 2 + i / 2], sel);
                    s[r] = __uint_as_float(i % 2 ? kscale[j][r][i / 2] & 0xFFFF0000u : kscale[j][r][i / 2] << 16);
                }
                const uint32_t a0[4] = {codes_f16<0>(w[0]), codes_f16<0>(w[1]), codes_f16<1>(w[0]), codes_f16<1>(w[1])};
                const uint32_t a1[4] = {codes_f16<2>(w[0]), codes_f16<2>(w[1]), codes_f16<3>(w[0]), codes_f16<3>(w[1])};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    mma16816<true>(d, a0, q[0][nt].x, q[0][nt].y);
                    mma16816<true>(d, a1, q[1][nt].x, q[1][nt].y);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[nt][j][e] = i == 0 ? d[e] * s[e >> 1] : fmaf(d[e], s[e >> 1], x[nt][j][e]);
                }
            }
        }
        // ---- the values into registers, and their slot free again
        if (!__all_sync(0xffffffffu, mbar_wait(&ms.v_full[warp][slot], phase, &ms.abort))) {
            ok = false;
            refetched = more;
            break;
        }
        uint32_t v[SUB][4][J / 2];
        float vs[SUB][2];  // of tokens g and g + 8
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                load_words<J / 2>(v[j][r], v_at + voff + ((r & 1) + 8 * (r >> 1) + 16 * j) * C::kRowBytes);
#pragma unroll
            for (int r = 0; r < 2; ++r) vs[j][r] = __uint_as_float(load_u16(vs_at + (16 * j + 8 * r + g) * 2) << 16);
        }
        __syncwarp();
        if (more)
            fetch(true, slot, zero_after(__float_as_uint(vs[SUB - 1][1]), nothing), base_next, ph_next);

        // ---- scores in base-2 units, masked
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < SUB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[nt][j][e] *= qscale[nt][e & 1];
        if constexpr (CAP) {
            const float cap_in = fminf(2.f * kLog2e / p.score_param, FLT_MAX),
                        cap_out = fminf(p.score_param * kLog2e, FLT_MAX);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < SUB; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[nt][j][e] = softcap_log2(x[nt][j][e], cap_in, cap_out);
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
        // ---- weights, and whether one exceeds what the reference allows
        float ref[SUB][2];
#pragma unroll
        for (int j = 0; j < SUB; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r) ref[j][r] = fmaxf(vs[j][r], kLeastRef);  // NaN: counts as the least
        float w[NT][SUB][4];
        bool raise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < SUB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[nt][j][e] = ex2_approx(x[nt][j][e] - m[nt][e & 1]);
                    raise |= w[nt][j][e] * ref[j][e >> 1] > 0x1p15f;
                }
        if (__any_sync(0xffffffffu, raise)) {
            float lr[SUB][2];
#pragma unroll
            for (int j = 0; j < SUB; ++j)
#pragma unroll
                for (int r = 0; r < 2; ++r) lr[j][r] = log2f(ref[j][r]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float alpha[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float top = -INFINITY;
#pragma unroll
                    for (int j = 0; j < SUB; ++j)
                        top = fmax3(top, x[nt][j][u] + lr[j][0], x[nt][j][u + 2] + lr[j][1]);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const float now = top > m[nt][u] + kRaise - 0.0625f ? top - kTop : m[nt][u];
                    alpha[u] = exp2f(m[nt][u] - now);
                    m[nt][u] = now;
                    l[nt][u] *= alpha[u];
                }
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    acc[nt][i][0] *= alpha[0];
                    acc[nt][i][1] *= alpha[1];
                    acc[nt][i][2] *= alpha[0];
                    acc[nt][i][3] *= alpha[1];
                }
#pragma unroll
                for (int j = 0; j < SUB; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[nt][j][e] = ex2_approx(x[nt][j][e] - m[nt][e & 1]);
            }
        }
        // ---- P, the sum of weights, and P^T as operand
        uint32_t pb[NT][SUB][2];
#pragma unroll
        for (int j = 0; j < SUB; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    l[nt][e & 1] += w[nt][j][e];
                    y[e] = w[nt][j][e] * vs[j][e >> 1];
                    // a token that the row does not keep, whatever its scale
                    if (!whole && x[nt][j][e] == -INFINITY) y[e] = 0.f;
                }
                pb[nt][j][0] = transpose8(pack_f16x2(y[0], y[1]));
                pb[nt][j][1] = transpose8(pack_f16x2(y[2], y[3]));
            }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int j = 0; j < SUB; ++j)
#pragma unroll
            for (int i = 0; i < J; ++i) {
                const uint32_t sel = i % 2 ? 0x7632u : 0x5410u;
                const uint32_t lo = prmt(v[j][0][i / 2], v[j][1][i / 2], sel), hi = prmt(v[j][2][i / 2], v[j][3][i / 2], sel);
                const uint32_t a0[4] = {codes_f16<0>(lo), codes_f16<1>(lo), codes_f16<0>(hi), codes_f16<1>(hi)};
                const uint32_t a1[4] = {codes_f16<2>(lo), codes_f16<3>(lo), codes_f16<2>(hi), codes_f16<3>(hi)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma16816<true>(acc[nt][2 * i], a0, pb[nt][j][0], pb[nt][j][1]);
                    mma16816<true>(acc[nt][2 * i + 1], a1, pb[nt][j][0], pb[nt][j][1]);
                }
            }
#pragma unroll
        for (int s = 0; s + 1 < ST; ++s) {
            base_of[s] = base_of[s + 1];
#pragma unroll
            for (int j = 0; j < SUB; ++j) ph[s][j] = ph[s + 1][j];
        }
        base_of[ST - 1] = base_next;
#pragma unroll
        for (int j = 0; j < SUB; ++j) ph[ST - 1][j] = ph_next[j];
        if (++slot == ST) {
            slot = 0;
            phase ^= 1u;
        }
        if (++at_step == sq.count || it + 1 == steps) {
            finish(at_step == sq.count);
            if (at_step == sq.count) {
                at_step = 0;
                entering = true;
                if (++pair == pairs_per_seq && it + 1 < steps) {
                    pair = 0;
                    sq = steps_of<C::kTokens>(p, __ldg(p.kv_lens + ++b));
                }
            }
        }
    }
    if (!ok) {
        // a copy did not arrive in time: report it, and give the copies still
        // under way the same time again before this CTA's shared memory is
        // given up
        ms.abort = 1;
        if (lane == 0) atomicExch(p.status, kDeviceTimeout);
        volatile int keep_waiting = 0;
        for (int s = 0; s < ST && it + s < steps; ++s) {
            const int at = (slot + s) % ST;
            const uint32_t par = phase ^ (slot + s >= ST ? 1u : 0u);
            mbar_wait(&ms.k_full[warp][at], par, &keep_waiting);
            mbar_wait(&ms.v_full[warp][at], par, &keep_waiting);
        }
        if (refetched) mbar_wait(&ms.k_full[warp][slot], phase ^ 1u, &keep_waiting);
    }
}

// The codes of the cache's keys or values as [pages * heads][page][D / 2] bytes:
// boxes of box_rows tokens.
template <int D>
bool make_codes_map(CUtensorMap *map, const void *base, const KvCache &c, int box_rows) {
    const uint64_t dims[3] = {D / 2, (uint64_t)c.page, (uint64_t)c.num_pages * c.H};
    const uint64_t strides[2] = {D / 2, (uint64_t)D / 2 * c.page};
    const uint32_t box[3] = {D / 2, (uint32_t)box_rows, 1};
    return make_tile_map_3d(map, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, strides, box,
                            D == 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
}

template <int D, int NT, bool CAP>
cudaError_t launch_cache4(const CacheAttnProblem &p, cudaStream_t stream) {
    using C = Cfg4<D, NT>;
    auto kernel = cache_attention_int4_kernel<D, NT, CAP>;
    const int row_tiles = (p.Q * p.G + C::kRows - 1) / C::kRows;
    const int64_t pairs = (int64_t)p.B * p.cache.H * row_tiles;
    if (pairs > INT_MAX) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int box_rows = p.cache.page < C::kTokens ? p.cache.page : C::kTokens;
    CUtensorMap map_k, map_v;
    if (!make_codes_map<D>(&map_k, p.cache.k, p.cache, box_rows) || !make_codes_map<D>(&map_v, p.cache.v, p.cache, box_rows))
        return cudaErrorInvalidValue;
    kernel<<<(unsigned)main_ctas(p, C::kTokens), kThreads, C::kSmem, stream>>>(map_k, map_v, p, row_tiles, box_rows);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_join<D, C::kRows, C::kTokens>(p, row_tiles, pairs, stream);
}

template <int D>
cudaError_t launch_cache4_rows(const CacheAttnProblem &p, cudaStream_t stream) {
    if (p.score_kind == FLEX_SCORE_SOFTCAP)
        return tile_rows(p) == 8 ? launch_cache4<D, 1, true>(p, stream) : launch_cache4<D, 2, true>(p, stream);
    return tile_rows(p) == 8 ? launch_cache4<D, 1, false>(p, stream) : launch_cache4<D, 2, false>(p, stream);
}

}  // namespace

int64_t cache_attention_int4_workspace(const CacheAttnProblem &p) {
    return workspace_partials(p.B) +
           2 * kWarps * main_ctas(p, Cfg4<128, 1>::kTokens) * partial_floats(tile_rows(p), p.cache.D) * 4;
}

cudaError_t launch_cache_attention_int4(const CacheAttnProblem &p, cudaStream_t stream) {
    return p.cache.D == 64 ? launch_cache4_rows<64>(p, stream) : launch_cache4_rows<128>(p, stream);
}

}  // namespace flex
