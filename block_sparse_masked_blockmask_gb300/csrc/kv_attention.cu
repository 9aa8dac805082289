// Attention of a sequence's newest tokens against its paged cache: for every
// query row (token t of Q, head h; position pos = kv_lens[b] - Q + t)
//   s[kv] = score_mod(scale q.k[kv])  for the kv its mask keeps, kv <= pos
//   out   = sum_kv exp(s[kv] - lse) v[kv],   lse = ln sum_kv exp(s[kv])
// in one pass over the keys (running maximum and sum), the query heads that
// share a key head reading it together.
//
// Bound by memory: the visible tokens' keys and values are read once (1 or 2
// bytes a value) for 4 G Q flops per pair of them.  Measured against the 6.77
// TB/s of a copy (32 sequences x 8 heads x 8192 tokens, D 128, e4m3, G 4): 93.4 us,
// 85%; bf16 of half the length 88.7 us, 89%; G 8: 82%; G 16, two row tiles: 75%.
// Above 16 rows per head the products bind (197 TFLOP/s at G 8, Q 64; bf16 149).
//
// The products run on mma.sync m16n8k16: one such tile has 16 keys against 8
// query rows, which is what a step of decoding has.  A tcgen05 tile has 128
// rows, and e4m3 keys would have to be written back to shared memory as 16-bit
// values to meet a bf16 query there, which costs more than the product.  At 6.8
// TB/s an SM receives 23 e4m3 values a clock; 8 rows of products on them are 375
// flops a clock.  What binds beside the memory is the work on the values:
// converting them (two codes in 2 cycles of a sub-partition, or 4 where they
// lie in a word's upper half), pairing them, and the latency of it all with
// two warps on a sub-partition.
//
//  * A step of a warp is 64 tokens of one head (32 of bf16 at D 128): keys and
//    values come by TMA (128-byte swizzle, so that the reads below are free of
//    bank conflicts) into the warp's own ring and go from there into registers
//    at once, which frees the slot for the next step while this one computes:
//    one slot in flight and one in registers (two slots of half the size: 101
//    us for 98, 64 sequences ragged to 8192).  Eight warps an SM, since twelve
//    leave 168 registers each, too few for this without spilling.
//  * Keys are the A operand of S^T = K Q^T: thread (g, t) of a warp (lane =
//    4 g + t) reads 16-byte pieces of keys g and g + 8, in a fixed permutation of
//    the head dim that Q's operand follows.  Values are the A operand of
//    O^T = V^T P^T: the thread reads the pieces at its own head dims of the
//    tokens 2t, 2t+1, 2t+8, 2t+9 and pairs them with byte permutes.
//  * e4m3 codes convert to fp16 exactly.  Q rows are divided by a power of two
//    first so that they fit fp16 (bf16 values keep all their bits down to 2^-14
//    of the row's largest).  The page's scale of K multiplies the scores, the
//    one of V the weights: P is kept relative to the largest V scale met, which
//    rescales the accumulators when it grows.  That reference is one for all rows
//    of a tile and goes by scales alone, so that a page with less than 2^-6 of it
//    would lose weights below fp16's smallest step to a page that a row may not
//    even keep: such a page's products are taken by themselves, 16 tokens at a
//    time, with the weights as they are, and scaled in float32.  P is rounded to
//    fp16 (11 bits), beside a bf16 cache to bf16 (8 bits) like the operands it
//    meets.
//  * S^T's accumulators hold keys along lanes' g and rows along t: after
//    exp, one 8 x 8 transpose (movmatrix) per 8 keys makes them the B operand
//    P^T.  Statistics, sums and accumulators are float32, and the sum takes the
//    unrounded weights.
//  * Weights are relative to 2^-7 of the largest when that was last raised, and it
//    is only raised when a score exceeds it by 2^8 (votes instead of reductions on
//    most steps): they stay below 2^15, and fp16's smallest step is 2^-31 of the
//    largest or less.  Small weights and pages with a small V scale beside
//    one with a large scale need the room below.
//  * The steps of all sequences, heads and row tiles form one list, which the
//    warps of one wave of CTAs share out evenly, so that ragged batches and a
//    few long sequences fill the SMs alike (an earlier form with a cluster of
//    CTAs for each took 108 and 116 us for what takes 98 and 96 now).  A warp
//    works alone: its ring runs on from one (sequence, head, row tile) to
//    the next, and no barrier joins it to other warps.  Where it covers all
//    steps of one it writes the rows; where a cut falls inside one, the pieces'
//    statistics and accumulators go to the workspace and a second, dependent
//    launch joins them.  Nothing is joined by atomics: results do not depend on
//    the order in which warps run.
//  * Only steps at an edge (the last tokens, a window's ends, a bad page)
//    evaluate the mask; there the values of tokens that no row keeps are
//    zeroed, so that whatever lies in those slots has no effect, and where
//    rows of the call differ in what they keep and such a token's value is not
//    finite, the step's product is done once per query token.  These steps and
//    those with a page of a small scale share one path, a head dim tile at a time,
//    so that it needs no second set of accumulators (with one: 116 bytes of spills
//    at 16 rows and D 128, and 115 us for 106 at G 16).
#include "kv_attention_common.cuh"

namespace flex {
namespace {

constexpr float kApart = 0x1p-6f;  // pages whose V scale is below this share of the largest are added apart

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

// D: head dim; E4M3: cache type (else bf16); NT: tiles of 8 query rows.
template <int D, bool E4M3, int NT>
struct Cfg {
    static constexpr int kElem = E4M3 ? 1 : 2;
    static constexpr int kRowBytes = D * kElem;
    static constexpr int kPanelBytes = kRowBytes < 128 ? kRowBytes : 128;  // a row of a staged panel (TMA swizzle span)
    static constexpr int kPanels = kRowBytes / kPanelBytes;
    // bytes of keys (of values) per step of a warp: 64 tokens at most
    static constexpr int kTile = NT == 1 && kRowBytes >= 128 ? 8192 : 4096;
    static constexpr int kTokens = kTile / kRowBytes;
    static constexpr int kSub = kTokens / 16;           // groups of 16 tokens per step
    static constexpr int kStages = 8192 / kTile;        // steps in flight per warp, beside the one in registers
    static constexpr int kSteps = D / 16;               // k16 steps of S, m16 tiles of O
    static constexpr int kKWords = kRowBytes / 16;      // words of one key a thread holds
    static constexpr int kVBytes = kRowBytes / 8;       // bytes of one value a thread holds
    static constexpr int kVLoad = kVBytes < 16 ? 8 : 16;
    static constexpr int kRows = 8 * NT;
    // shared memory of a warp: its ring and its Q operand
    static constexpr int kRing = kStages * 2 * kTile;
    static constexpr int kQBytes = NT * kSteps * 32 * 8;
    static constexpr int kSmem = 1024 + kWarps * (kRing + kQBytes);  // 1024: alignment of the swizzle
};

struct Misc {
    uint64_t k_full[kWarps][2], v_full[kWarps][2];
    int64_t sums[kWarps];
    int abort;
};

// CAP: softcap scores, compiled apart: their instructions in the loop's body, which
// outgrows the instruction caches near the warps, cost the other scores 1% (64
// sequences ragged to 8192: 98.5 us for 97.4).
template <int D, bool E4M3, int NT, bool CAP>
__global__ void __launch_bounds__(kThreads, 2)
    cache_attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                           const CacheAttnProblem p, int row_tiles, int box_rows) {
    using C = Cfg<D, E4M3, NT>;
    constexpr int SUB = C::kSub, KS = C::kSteps, ST = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Misc ms;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023)) +
                    warp * C::kRing;
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
    // 32 k + i, so that the loads' latencies are met once in 32 steps: its first
    // token, and of its 16-token groups page * heads + head, or -1 where there
    // is nothing that a row keeps, and the page's scales.  The groups of one box
    // share a page.
    int look_b = b;
    int64_t look_off = off;
    int looked = 0;
    int base_lane = 0, ph_lane[SUB];
    float ks_lane[SUB], vs_lane[SUB];
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
        // the next batch begins where lane 31's successor would be
        look_b = __shfl_sync(0xffffffffu, lb, 31);
        look_off = __shfl_sync(0xffffffffu, lo_, 31) + 1;
        looked += 32;
    };
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
    // of the current step and the ST - 1 behind it
    int base_of[ST], ph[ST][SUB];
    float ks[ST][SUB], vs[ST][SUB];
    auto take_place = [&](int i, int &base, int (&to)[SUB]) {
        base = __shfl_sync(0xffffffffu, base_lane, i);
#pragma unroll
        for (int j = 0; j < SUB; ++j) to[j] = __shfl_sync(0xffffffffu, ph_lane[j], i);
    };
    auto take_scales = [&](int i, float (&k)[SUB], float (&v)[SUB]) {
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
            k[j] = E4M3 ? __shfl_sync(0xffffffffu, ks_lane[j], i) : 1.f;
            v[j] = E4M3 ? __shfl_sync(0xffffffffu, vs_lane[j], i) : 1.f;
        }
    };
    lookup();
#pragma unroll
    for (int s = 0; s < ST; ++s) {
        take_place(s, base_of[s], ph[s]);
        if (s < steps) {
            uint8_t *dst = ring + s * 2 * C::kTile;
            fetch(&map_k, dst, &ms.k_full[warp][s], base_of[s], ph[s]);
            fetch(&map_v, dst + C::kTile, &ms.v_full[warp][s], base_of[s], ph[s]);
        }
    }
#pragma unroll
    for (int s = 0; s < ST; ++s) take_scales(s, ks[s], vs[s]);

    const uint32_t nothing = (uint32_t)p.cache.page & 1u;  // 0, which the compiler does not know
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

    // ---- the pair being computed
    Steps sq = steps_of<C::kTokens>(p, __ldg(p.kv_lens + b));
    int pair = (int)(off / sq.count), at_step = (int)(off % sq.count);
    bool entering = true, whole_start = false;
    int hk = 0, r0 = 0, r1 = 0, tmin = 0, tmax = 0, n = 0, hi = 0, send = 0, all_hi = 0;
    int lo_min = 0, all_lo = 0;
    float slope[NT][2], qscale[NT][2];  // of this thread's rows, columns 2t and 2t + 1 of each row tile (base-2 units)
    int pos[NT][2], seen[NT][2];        // position, and the last kv it keeps (-1: nothing)
    float m[NT][2], l[NT][2], acc[NT][KS][4], vref = 0.f;
    uint2 *qs = reinterpret_cast<uint2 *>(ring - warp * C::kRing + kWarps * C::kRing + warp * C::kQBytes);

    // ---- the end of a piece: the pair's rows where the warp covered all of its
    // steps, else a partial result
    auto finish = [&](bool whole_end) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[nt][u] += __shfl_xor_sync(0xffffffffu, l[nt][u], o);
        const float f = E4M3 ? vref : 1.f;
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
                    const int d = E4M3 ? g * (D / 8) + 2 * i : (i / 4) * 64 + g * 8 + 2 * (i % 4);
                    const float a = acc[nt][i][u] * f, z = acc[nt][i][u + 2] * f;
                    if (whole_start && whole_end)
                        store_pair<D>(p, b, hk, r0 + r, d, a, z, m[nt][u], l[nt][u]);
                    else
                        *reinterpret_cast<float2 *>(part + r * D + d) = make_float2(a, z);
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
            tmin = r0 / p.G;
            tmax = r1 / p.G;
            // what any row of the tile keeps: [0, send) and [lo_min, hi)
            hi = p.causal ? max(n - p.Q + tmax + 1, 0) : n;
            lo_min = p.causal ? (int)max((int64_t)n - p.Q + tmin - p.window + 1, (int64_t)0) : 0;
            send = min(p.sinks, hi);
            // what every row keeps, for steps without mask work
            all_hi = p.causal ? n - p.Q + tmin + 1 : (n - p.Q + tmin >= 0 ? n : 0);
            all_lo = p.causal ? (int)max((int64_t)n - p.Q + tmax - p.window + 1, (int64_t)0) : 0;
            // Q operand: lane (g, t) takes row g at the head dims of its key words
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = r0 + nt * 8 + g;
                const bool live = row <= r1;
                const uint16_t *src = p.q + b * p.q_stride[0] +
                                      (int64_t)(hk * p.G + (live ? row % p.G : 0)) * p.q_stride[1] +
                                      (int64_t)(live ? row / p.G : 0) * p.q_stride[2];
                uint2 w[KS];
#pragma unroll
                for (int s = 0; s < KS; s += 2) {  // 16 bytes: two steps
                    const int d = C::kPanelBytes == 64 ? t * 16 + s * 4
                                  : E4M3               ? (2 * t + s / 4) * 16 + (s % 4) * 4
                                                       : (s / 4) * 64 + (2 * t + (s % 4) / 2) * 8;
                    const uint4 v = live ? *reinterpret_cast<const uint4 *>(src + d) : make_uint4(0, 0, 0, 0);
                    w[s] = make_uint2(v.x, v.y);
                    w[s + 1] = make_uint2(v.z, v.w);
                }
                float qf = 1.f;
                if constexpr (E4M3) {
                    uint32_t top = 0u;
#pragma unroll
                    for (int s = 0; s < KS; ++s)
                        top = max(max(top, max(w[s].x & 0x7FFFu, (w[s].x >> 16) & 0x7FFFu)),
                                  max(w[s].y & 0x7FFFu, (w[s].y >> 16) & 0x7FFFu));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // the power of two of the row's largest magnitude; 1 for a
                    // row of zeros and for rows with infinities or NaN, whose
                    // scores are not finite
                    const uint32_t e = top >> 7;
                    qf = e == 0u || e == 255u ? 1.f : __uint_as_float(e << 23);
                    const float f = 1.f / qf;
#pragma unroll
                    for (int s = 0; s < KS; ++s) {
                        w[s].x = pack_f16x2(__uint_as_float(w[s].x << 16) * f, __uint_as_float(w[s].x & 0xFFFF0000u) * f);
                        w[s].y = pack_f16x2(__uint_as_float(w[s].y << 16) * f, __uint_as_float(w[s].y & 0xFFFF0000u) * f);
                    }
                }
#pragma unroll
                for (int s = 0; s < KS; ++s) qs[(nt * KS + s) * 32 + lane] = w[s];  // read back by this lane alone
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
            vref = 0.f;
        }
        const int base = base_of[0];
        const bool more = it + ST < steps;
        int base_next, ph_next[SUB];
        float ks_next[SUB], vs_next[SUB];
        if (more && it + ST == looked) lookup();
        take_place((it + ST) % 32, base_next, ph_next);
        take_scales((it + ST) % 32, ks_next, vs_next);
        bool whole = base + C::kTokens <= all_hi && (base >= all_lo || base + C::kTokens <= p.sinks);
#pragma unroll
        for (int j = 0; j < SUB; ++j) whole = whole && ph[0][j] >= 0;
        // the largest V scale here; pages far below the largest of all are added
        // apart (see the products), in steps that take the longer way like those
        // at an edge
        float vmax = vs[0][0];
#pragma unroll
        for (int j = 1; j < SUB; ++j) vmax = fmaxf(vmax, vs[0][j]);
        bool apart = false;
        if constexpr (E4M3) {
            const float least = fmaxf(vref, vmax) * kApart;
#pragma unroll
            for (int j = 0; j < SUB; ++j) apart |= vs[0][j] > 0.f && vs[0][j] < least;
            whole = whole && !apart;
        }
        const uint32_t k_at = ring_at + slot * 2 * C::kTile, v_at = k_at + C::kTile;
        // ---- S^T = K Q^T
        if (!__all_sync(0xffffffffu, mbar_wait(&ms.k_full[warp][slot], phase, &ms.abort))) {
            ok = false;
            break;
        }
        uint32_t kw[SUB][2][C::kKWords];
#pragma unroll
        for (int j = 0; j < SUB; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int c = 0; c < C::kKWords / 4; ++c)
                    load_shared<16>(&kw[j][r][4 * c], k_at + koff[c & 1] + (c >> 1) * C::kTokens * C::kPanelBytes +
                                                          (16 * j + 8 * r) * C::kPanelBytes);
        __syncwarp();
        if (more)  // the slot is free as soon as its words are in registers
            fetch(&map_k, ring + slot * 2 * C::kTile + zero_after(kw[SUB - 1][1][C::kKWords - 1], nothing),
                  &ms.k_full[warp][slot], base_next, ph_next);
        float x[NT][SUB][4];
#pragma unroll
        for (int j = 0; j < SUB; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) x[nt][j][0] = x[nt][j][1] = x[nt][j][2] = x[nt][j][3] = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            uint2 q[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) q[nt] = qs[(nt * KS + s) * 32 + lane];
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                uint32_t a[4];
                if constexpr (E4M3) {
                    a[0] = e4m3_lo(kw[j][0][s]);
                    a[1] = e4m3_lo(kw[j][1][s]);
                    a[2] = e4m3_hi(kw[j][0][s]);
                    a[3] = e4m3_hi(kw[j][1][s]);
                } else {
                    a[0] = kw[j][0][2 * s];
                    a[1] = kw[j][1][2 * s];
                    a[2] = kw[j][0][2 * s + 1];
                    a[3] = kw[j][1][2 * s + 1];
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma16816<E4M3>(x[nt][j], a, q[nt].x, q[nt].y);
            }
        }
        // ---- the values into registers, and their slot free again
        if (!__all_sync(0xffffffffu, mbar_wait(&ms.v_full[warp][slot], phase, &ms.abort))) {
            ok = false;
            refetched = more;
            break;
        }
        uint32_t v[SUB][4][C::kVBytes / 4];
#pragma unroll
        for (int j = 0; j < SUB; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < C::kVBytes / C::kVLoad; ++c)
                    load_shared<C::kVLoad>(&v[j][r][c * 4], v_at + voff[r & 1] + c * C::kTokens * C::kPanelBytes +
                                                                (16 * j + 8 * (r >> 1)) * C::kPanelBytes);
        __syncwarp();
        if (more)
            fetch(&map_v, ring + slot * 2 * C::kTile + C::kTile + zero_after(v[SUB - 1][3][C::kVBytes / 4 - 1], nothing),
                  &ms.v_full[warp][slot], base_next, ph_next);

        // ---- scores in base-2 units, masked
        float top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < SUB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[nt][j][e] *= qscale[nt][e & 1] * ks[0][j];
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
                    const float now = w > m[nt][u] + kRaise ? w - kTop : m[nt][u];
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
            const float vf = !E4M3 || apart || vs[0][j] == vref ? 1.f : vs[0][j] / vref;
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
        // operand of head dim tile i from the values of 16 tokens
        auto operand = [&](int j, int i, auto &&value, uint32_t (&a)[4]) {
            if constexpr (E4M3) {
                const uint32_t sel = i & 1 ? 0x7362u : 0x5140u;
                const uint32_t lo2 = prmt(value(j, 0, i / 2), value(j, 1, i / 2), sel);
                const uint32_t hi2 = prmt(value(j, 2, i / 2), value(j, 3, i / 2), sel);
                a[0] = e4m3_lo(lo2);
                a[1] = e4m3_hi(lo2);
                a[2] = e4m3_lo(hi2);
                a[3] = e4m3_hi(hi2);
            } else {
                a[0] = prmt(value(j, 0, i), value(j, 1, i), 0x5410u);
                a[1] = prmt(value(j, 0, i), value(j, 1, i), 0x7632u);
                a[2] = prmt(value(j, 2, i), value(j, 3, i), 0x5410u);
                a[3] = prmt(value(j, 2, i), value(j, 3, i), 0x7632u);
            }
        };
        bool plain = true, mixed = false;  // mixed: a token that some rows keep and some do not has a value that is not finite
        if (!whole) {
            // values of tokens that no row keeps: zero, whatever lies there
#pragma unroll
            for (int j = 0; j < SUB; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int kv = base + 16 * j + 2 * t + (r & 1) + (r >> 1) * 8;
                    const bool any = ph[0][j] >= 0 && kv < hi && (kv >= lo_min || kv < send);
                    const bool every = kv < all_hi && (kv >= all_lo || kv < p.sinks);
                    bool odd = false;
#pragma unroll
                    for (int c = 0; c < C::kVBytes / 4; ++c) {
                        if (!any) v[j][r][c] = 0u;
                        if constexpr (E4M3)
                            odd |= __vcmpeq4(v[j][r][c] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0u;
                        else
                            odd |= __vcmpgeu2(v[j][r][c] & 0x7FFF7FFFu, 0x7F807F80u) != 0u;
                    }
                    mixed |= odd && !every;
                }
            mixed = __any_sync(0xffffffffu, mixed);
            plain = !mixed && !apart;
        }
        if (plain) {
#pragma unroll
            for (int j = 0; j < SUB; ++j)
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    uint32_t a[4];
                    operand(j, i, [&](int j, int r, int c) { return v[j][r][c]; }, a);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816<E4M3>(acc[nt][i], a, pb[nt][j][0], pb[nt][j][1]);
                }
        } else {
            // mixed: one query token's rows at a time, with what they do not
            // keep zeroed; the other rows' columns keep their sums, since their
            // zero weights must not meet a value that is not finite either.
            // apart: weights as they are, products of 16 tokens by themselves,
            // which take their page's scale in float32
#pragma unroll 1
            for (int tok = tmin; tok <= (mixed ? tmax : tmin); ++tok) {
                const int at = n - p.Q + tok;
                auto value = [&](int j, int r, int c) {
                    const int kv = base + 16 * j + 2 * t + (r & 1) + (r >> 1) * 8;
                    const bool keep = p.causal ? kv <= at && (at - kv < p.window || kv < p.sinks) : at >= 0 && kv < n;
                    return !mixed || keep ? v[j][r][c] : 0u;
                };
                auto weight = [&](int nt, int j, int e) {  // the operand's column is the lane's g
                    return !mixed || (r0 + nt * 8 + g) / p.G == tok ? pb[nt][j][e] : 0u;
                };
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    float sum[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum[nt][e] = acc[nt][i][e];
#pragma unroll
                    for (int j = 0; j < SUB; ++j) {
                        uint32_t a[4];
                        operand(j, i, value, a);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (!apart) {
                                mma16816<E4M3>(sum[nt], a, weight(nt, j, 0), weight(nt, j, 1));
                            } else {
                                float part[4] = {0.f, 0.f, 0.f, 0.f};
                                mma16816<E4M3>(part, a, weight(nt, j, 0), weight(nt, j, 1));
#pragma unroll
                                for (int e = 0; e < 4; ++e) sum[nt][e] += part[e] * (vs[0][j] / vref);
                            }
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!mixed || (r0 + nt * 8 + 2 * t + (e & 1)) / p.G == tok) acc[nt][i][e] = sum[nt][e];
                }
            }
        }
#pragma unroll
        for (int s = 0; s + 1 < ST; ++s) {
            base_of[s] = base_of[s + 1];
#pragma unroll
            for (int j = 0; j < SUB; ++j) ph[s][j] = ph[s + 1][j], ks[s][j] = ks[s + 1][j], vs[s][j] = vs[s + 1][j];
        }
        base_of[ST - 1] = base_next;
#pragma unroll
        for (int j = 0; j < SUB; ++j) ph[ST - 1][j] = ph_next[j], ks[ST - 1][j] = ks_next[j], vs[ST - 1][j] = vs_next[j];
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

template <int D, bool E4M3, int NT, bool CAP>
cudaError_t launch_cache(const CacheAttnProblem &p, cudaStream_t stream) {
    using C = Cfg<D, E4M3, NT>;
    auto kernel = cache_attention_kernel<D, E4M3, NT, CAP>;
    const int row_tiles = (p.Q * p.G + C::kRows - 1) / C::kRows;
    const int64_t pairs = (int64_t)p.B * p.cache.H * row_tiles;
    if (pairs > INT_MAX) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int box_rows = p.cache.page < C::kTokens ? p.cache.page : C::kTokens;
    CUtensorMap map_k, map_v;
    if (!make_cache_map<D, E4M3>(&map_k, p.cache.k, p.cache, box_rows) ||
        !make_cache_map<D, E4M3>(&map_v, p.cache.v, p.cache, box_rows))
        return cudaErrorInvalidValue;
    kernel<<<(unsigned)main_ctas(p, C::kTokens), kThreads, C::kSmem, stream>>>(map_k, map_v, p, row_tiles, box_rows);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_join<D, C::kRows, C::kTokens>(p, row_tiles, pairs, stream);
}

template <int D, bool E4M3>
cudaError_t launch_cache_rows(const CacheAttnProblem &p, cudaStream_t stream) {
    if (p.score_kind == FLEX_SCORE_SOFTCAP)
        return tile_rows(p) == 8 ? launch_cache<D, E4M3, 1, true>(p, stream) : launch_cache<D, E4M3, 2, true>(p, stream);
    return tile_rows(p) == 8 ? launch_cache<D, E4M3, 1, false>(p, stream) : launch_cache<D, E4M3, 2, false>(p, stream);
}

int step_tokens(const CacheAttnProblem &p, int cache_dtype) {
    const int row = p.cache.D * (cache_dtype == FLEX_DTYPE_E4M3 ? 1 : 2);
    return (tile_rows(p) == 8 && row >= 128 ? 8192 : 4096) / row;
}

}  // namespace

int64_t cache_attention_workspace(const CacheAttnProblem &p, int cache_dtype) {
    if (cache_dtype == FLEX_DTYPE_INT4) return cache_attention_int4_workspace(p);
    return workspace_partials(p.B) +
           2 * kWarps * main_ctas(p, step_tokens(p, cache_dtype)) * partial_floats(tile_rows(p), p.cache.D) * 4;
}

cudaError_t launch_cache_attention(const CacheAttnProblem &p, int cache_dtype, cudaStream_t stream) {
    if (cache_dtype == FLEX_DTYPE_INT4) return launch_cache_attention_int4(p, stream);
    if (cache_dtype == FLEX_DTYPE_E4M3)
        return p.cache.D == 64 ? launch_cache_rows<64, true>(p, stream) : launch_cache_rows<128, true>(p, stream);
    return p.cache.D == 64 ? launch_cache_rows<64, false>(p, stream) : launch_cache_rows<128, false>(p, stream);
}

}  // namespace flex
