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
#include <cfloat>
#include <climits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_internal.h"
#include "ptx.cuh"

namespace flex {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kJoinThreads = 512;
constexpr int kJoinMany = 8;       // warps of the main launch per pair, from which CTAs join a row
constexpr int kMaxCtas = 152 * 2;  // of the main launch: two on every SM
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Entering and finishing a (sequence, head, row tile) costs a warp the time of
// some steps: the list counts that many units more for each (512 pairs, ragged
// to 8192 tokens: none 134 us, 1: 114, 2 to 6: 98).  A warp takes one unit at
// least: few steps are over sooner with more of them in flight (513 tokens of 8
// heads: 12.5 us, and 14.6 with two, 18.1 with four).
constexpr int kEnterCost = 3;
constexpr int kMinShare = 1;
constexpr float kTop = 7.f;     // raising the reference leaves the largest weight at 2^7
constexpr float kRaise = 15.f;  // and is due when one would pass 2^15
constexpr float kApart = 0x1p-6f;  // pages whose V scale is below this share of the largest are added apart

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
// cap tanh(u), u = s / cap, in base-2 units.  From |u| = 1/4 on as cap (1 - 2 / (1
// + e^(2 u))), which is within 2^-22 cap: about 2^-20 of the result, but nothing
// of it where u is small.  There the Taylor series to u^9, which leaves out less
// than 2^-26 of it.  Together a tenth of tanhf's instructions.
// in = 2 log2(e) / cap, out = cap log2(e), both finite.
__device__ __forceinline__ float softcap_log2(float s, float in, float out) {
    constexpr double k = 0.69314718055994530942 * 0.69314718055994530942 / 4;  // u^2 = k z^2
    const float z = s * in, t = z * z;
    float near = fmaf(t, (float)(62. / 2835 * k * k * k * k), (float)(-17. / 315 * k * k * k));
    near = fmaf(t, near, (float)(2. / 15 * k * k));
    near = fmaf(t, near, (float)(-1. / 3 * k));
    near = fmaf(t, near, 1.f) * (s * kLog2e);
    const float far = fmaf(out, -2.f * rcp_approx(1.f + ex2_approx(z)), out);
    return fabsf(z) < 0.5f * kLog2e ? near : far;
}
// 8 x 8 transpose of 16-bit values across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Zero, once the loads that a depends on have returned (a warp's loads from
// shared memory return in order): a slot is refilled only after its last word
// was read.  The bit test cannot be folded away, and lane 0 alone uses it.
__device__ __forceinline__ uint32_t zero_after(uint32_t a, uint32_t zero) { return a & zero; }

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

// Steps of a sequence: tokens that any of its query rows keeps, [0, send) and
// [lo_min, hi), in whole steps.
struct Steps {
    int n, hi, send, lo, nsink, count;
    int64_t lo_min;
    __device__ __forceinline__ int base(int i, int tokens) const {
        return i < nsink ? i * tokens : lo + (i - nsink) * tokens;
    }
};
template <int TOKENS>
__device__ __forceinline__ Steps steps_of(const CacheAttnProblem &p, int kv_len) {
    Steps s;
    s.n = (int)min((int64_t)max(kv_len, 0), (int64_t)p.max_pages * p.cache.page);
    s.hi = s.n;  // the last query token is the last token
    s.lo_min = p.causal ? max((int64_t)s.n - p.Q - p.window + 1, (int64_t)0) : 0;
    s.lo = (int)min(s.lo_min, (int64_t)s.hi) / TOKENS * TOKENS;
    s.send = min(p.sinks, s.hi);
    s.nsink = (s.send + TOKENS - 1) / TOKENS;
    if (s.nsink * (int64_t)TOKENS >= s.lo) {
        s.nsink = 0;
        s.lo = 0;
    }
    s.count = max(s.nsink + (s.hi - s.lo + TOKENS - 1) / TOKENS, 1);  // an empty sequence: one empty step
    return s;
}

// The workspace: the size of a warp's share of the list, where each sequence
// begins in it, and two partial results per warp (rows x (D + 2) floats:
// accumulators, maximum, sum): of a piece that begins inside its (sequence,
// head, row tile), and of one that begins with it but does not end it.
__host__ __device__ constexpr int64_t workspace_partials(int64_t B) { return (8 * (B + 1) + 15) / 16 * 16; }
__host__ __device__ constexpr int64_t partial_floats(int rows, int D) { return (int64_t)rows * (D + 2); }

// Two neighbouring output values of query row `row` of a head group, and its lse.
template <int D>
__device__ __forceinline__ void store_pair(const CacheAttnProblem &p, int b, int hk, int row, int d, float a, float z,
                                           float top, float sum) {
    const int64_t o = ((int64_t)b * p.Hq + hk * p.G + row % p.G) * p.Q + row / p.G;
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);  // NaN stays
    *reinterpret_cast<uint32_t *>(p.out + o * D + d) = pack_bf16x2(a * inv, z * inv);
    if (d == 0) p.lse[o] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

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

    // ---- the warp's share of the list.  Thread i adds up a run of sequences;
    // the block's prefix sums then give the total and where a step falls.
    const int pairs_per_seq = p.cache.H * row_tiles;  // (head, row tile) pairs, the row tiles innermost
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b_first = min((int)threadIdx.x * per, p.B), b_last = min(b_first + per, p.B);
    auto seq_units = [&](int i) {
        return (int64_t)(steps_of<C::kTokens>(p, __ldg(p.kv_lens + i)).count + kEnterCost) * pairs_per_seq;
    };
    int64_t mine = 0;
    for (int i = b_first; i < b_last; ++i) mine += seq_units(i);
    int64_t upto = mine;  // inclusive scan
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) ms.sums[warp] = upto;
    __syncthreads();
    int64_t total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += ms.sums[w];
        total += ms.sums[w];
    }
    const int64_t workers = (int64_t)gridDim.x * kWarps;
    const int64_t share = max((total + workers - 1) / workers, (int64_t)kMinShare);
    int64_t *head = reinterpret_cast<int64_t *>(p.workspace);
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) head[0] = share;
        int64_t at = before + upto - mine;
        for (int i = b_first; i < b_last; ++i) {
            head[1 + i] = at;
            at += seq_units(i);
        }
    }
    // neighbouring shares go to different CTAs, so that few steps spread over
    // the SMs
    const int worker = warp * (int)gridDim.x + (int)blockIdx.x;
    const int64_t begin = worker * share;
    if (begin >= total) return;
    // the sequence that `begin` falls in: first the block's warp, then its lane, then its run
    int b = 0;
    int64_t off = begin;
    {
        int64_t skipped = 0;
        int w0 = 0;
        while (w0 + 1 < kWarps && begin >= skipped + ms.sums[w0]) skipped += ms.sums[w0++];
        off = begin - skipped;
        b = w0 * 32 * per;
        for (int i0 = 0; i0 < 32 * per; i0 += 32) {  // 32 sequences at a time
            const int64_t size = b + lane < p.B ? seq_units(b + lane) : 0;
            int64_t sum = size;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            const unsigned past = __ballot_sync(0xffffffffu, sum > off);
            if (past) {
                const int f = __ffs(past) - 1;
                off -= __shfl_sync(0xffffffffu, sum - size, f);
                b += f;
                break;
            }
            off -= __shfl_sync(0xffffffffu, sum, 31);
            b += 32;
        }
    }

    // from units of the list to the steps among them: those of this warp, and
    // the first of them within its sequence
    int steps = 0;
    {
        int64_t left = min(share, total - begin), from = off;
        for (int i = b; left > 0; ++i) {
            const int count = steps_of<C::kTokens>(p, __ldg(p.kv_lens + i)).count, unit = count + kEnterCost;
            auto real = [&](int64_t o) { return o / unit * count + max((int)(o % unit) - kEnterCost, 0); };
            const int64_t to = min(from + left, (int64_t)unit * pairs_per_seq);
            const int64_t here = real(to) - real(from);
            if (steps == 0) {
                b = i;
                off = real(from);
            }
            steps += (int)here;
            left -= to - from;
            from = 0;
        }
    }
    if (steps == 0) return;

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

// Joins the pieces of one (sequence, head, row tile), one warp a row; nothing
// to do for one that a single warp covered.  For lists in which a pair is a few
// warps' share (512 pairs: 98 us in all, 137 with the kernel below).
template <int D, int ROWS, int TOKENS>
__global__ void __launch_bounds__(32 * ROWS) cache_attention_join_few_kernel(const CacheAttnProblem p, int row_tiles) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int V = D / 32;  // values per lane
    const int pairs_per_seq = p.cache.H * row_tiles;
    const int b = (int)(blockIdx.x / pairs_per_seq), pair = (int)(blockIdx.x % pairs_per_seq);
    const int r = threadIdx.x / 32, d = threadIdx.x % 32 * V, r0 = pair % row_tiles * ROWS;
    if (r0 + r >= p.Q * p.G) return;
    const int64_t *head = reinterpret_cast<const int64_t *>(p.workspace);
    const int64_t share = head[0];
    const int count = steps_of<TOKENS>(p, __ldg(p.kv_lens + b)).count;
    const int64_t begin = head[1 + b] + (int64_t)pair * (count + kEnterCost) + kEnterCost;  // of its first step
    const int c0 = (int)(begin / share), c1 = (int)((begin + count - 1) / share);
    if (c0 == c1) return;
    const float *parts =
        reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(p.workspace) + workspace_partials(p.B));
    float top = -FLT_MAX, sum = 0.f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    constexpr int U = 4;  // pieces in flight
    for (int c = c0; c <= c1; c += U) {
        float2 ml[U];
        float o[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ml[u] = make_float2(-FLT_MAX, 0.f);
#pragma unroll
            for (int v = 0; v < V; ++v) o[u][v] = 0.f;
            if (c + u <= c1) {
                const float *part = parts + (2 * (int64_t)(c + u) + (c + u == c0)) * partial_floats(ROWS, D);
                ml[u] = __ldcg(reinterpret_cast<const float2 *>(part + ROWS * D + 2 * r));
#pragma unroll
                for (int v = 0; v < V; v += 2) {
                    const float2 w = __ldcg(reinterpret_cast<const float2 *>(part + r * D + d + v));
                    o[u][v] = w.x;
                    o[u][v + 1] = w.y;
                }
            }
        }
        float now = top;
#pragma unroll
        for (int u = 0; u < U; ++u) now = fmaxf(now, ml[u].x);
        const float f0 = exp2f(top - now);
        top = now;
        sum *= f0;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] *= f0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float f = exp2f(ml[u].x - now);
            sum += f * ml[u].y;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] += f * o[u][v];
        }
    }
#pragma unroll
    for (int v = 0; v < V; v += 2)
        store_pair<D>(p, b, pair / row_tiles, r0 + r, d + v, acc[v], acc[v + 1], top, sum);
}

// The same for pairs that many warps share: one CTA for 32 head dims of a row,
// two of them a thread, in groups that share out the pieces (16 pairs of 76
// pieces: 96 us in all, 109 with the kernel above).
template <int D, int ROWS, int TOKENS>
__global__ void __launch_bounds__(kJoinThreads) cache_attention_join_kernel(const CacheAttnProblem p, int row_tiles) {
    constexpr int kColumns = 16, kGroups = kJoinThreads / kColumns, kJoinWarps = kJoinThreads / 32;
    __shared__ float top_s[kJoinWarps], sum_s[kJoinWarps], factor[kMaxCtas * kWarps];
    __shared__ float2 value_s[kJoinWarps][kColumns];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int pairs_per_seq = p.cache.H * row_tiles, warp = threadIdx.x / 32;
    const int b = (int)(blockIdx.x / pairs_per_seq), pair = (int)(blockIdx.x % pairs_per_seq), r = (int)blockIdx.y;
    const int64_t *head = reinterpret_cast<const int64_t *>(p.workspace);
    const int64_t share = head[0];
    const int count = steps_of<TOKENS>(p, __ldg(p.kv_lens + b)).count;
    const int64_t begin = head[1 + b] + (int64_t)pair * (count + kEnterCost) + kEnterCost;  // of its first step
    const int c0 = (int)(begin / share), c1 = (int)((begin + count - 1) / share);
    const int r0 = pair % row_tiles * ROWS;
    if (c0 == c1 || r0 + r >= p.Q * p.G) return;
    const float *parts =
        reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(p.workspace) + workspace_partials(p.B));
    auto part = [&](int c) { return parts + (2 * (int64_t)c + (c == c0)) * partial_floats(ROWS, D); };
    auto stats = [&](int c) { return __ldcg(reinterpret_cast<const float2 *>(part(c) + ROWS * D + 2 * r)); };
    // the pieces' maxima, and what each is worth relative to the largest
    const int pieces = c1 - c0 + 1;
    float top = -FLT_MAX;
    for (int c = threadIdx.x; c < pieces; c += kJoinThreads) {
        factor[c] = stats(c0 + c).x;
        top = fmaxf(top, factor[c]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (threadIdx.x % 32 == 0) top_s[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, top_s[w]);
    float sum = 0.f;
    for (int c = threadIdx.x; c < pieces; c += kJoinThreads) {
        factor[c] = exp2f(factor[c] - top);
        sum += factor[c] * stats(c0 + c).y;
    }
    __syncthreads();
    const int column = threadIdx.x % kColumns, group = threadIdx.x / kColumns;
    const int d = (int)blockIdx.z * 2 * kColumns + 2 * column;
    float2 s = make_float2(0.f, 0.f);
#pragma unroll 8
    for (int c = group; c < pieces; c += kGroups) {
        const float2 o = __ldcg(reinterpret_cast<const float2 *>(part(c0 + c) + r * D + d));
        s.x += o.x * factor[c];
        s.y += o.y * factor[c];
    }
    // over the threads: the row's sum, and each column's values
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    s.x += __shfl_xor_sync(0xffffffffu, s.x, kColumns);
    s.y += __shfl_xor_sync(0xffffffffu, s.y, kColumns);
    if (threadIdx.x % 32 == 0) sum_s[warp] = sum;
    if (threadIdx.x % 32 < kColumns) value_s[warp][column] = s;
    __syncthreads();
    if (threadIdx.x >= kColumns) return;
    sum = 0.f;
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        sum += sum_s[w];
        s.x += value_s[w][column].x;
        s.y += value_s[w][column].y;
    }
    store_pair<D>(p, b, pair / row_tiles, r0 + r, d, s.x, s.y, top, sum);
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

// Query rows per tile: 8, or 16 from nine rows on (the keys are converted once
// for both halves).
int tile_rows(const CacheAttnProblem &p) { return (int64_t)p.Q * p.G <= 8 ? 8 : 16; }

// CTAs of the main launch: one wave, or as many as there can be steps, from
// what the host knows of the lengths.
int64_t main_ctas(const CacheAttnProblem &p, int tokens) {
    const int rows = tile_rows(p);
    const int64_t pairs = (int64_t)p.B * p.cache.H * (((int64_t)p.Q * p.G + rows - 1) / rows);
    int64_t most = (int64_t)p.max_pages * p.cache.page;
    if (p.window != INT_MAX) {
        const int64_t w = (int64_t)p.window + p.sinks + p.Q + 2 * tokens;
        most = most < w ? most : w;
    }
    const int64_t steps = pairs * ((most + tokens - 1) / tokens + 1), wave = kMaxCtas;
    return steps < wave ? steps : wave;
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
    // the join is launched while the main kernel runs and waits for its end on
    // the device, which hides its launch
    cudaLaunchConfig_t cfg = {};
    const bool many = main_ctas(p, C::kTokens) * kWarps >= pairs * kJoinMany;
    const int live = (int)((int64_t)p.Q * p.G < C::kRows ? (int64_t)p.Q * p.G : C::kRows);
    cfg.gridDim = dim3((unsigned)pairs, many ? live : 1, many ? D / 32 : 1);
    cfg.blockDim = dim3(many ? kJoinThreads : 32 * C::kRows);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return many ? cudaLaunchKernelEx(&cfg, cache_attention_join_kernel<D, C::kRows, C::kTokens>, p, row_tiles)
                : cudaLaunchKernelEx(&cfg, cache_attention_join_few_kernel<D, C::kRows, C::kTokens>, p, row_tiles);
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
    return workspace_partials(p.B) +
           2 * kWarps * main_ctas(p, step_tokens(p, cache_dtype)) * partial_floats(tile_rows(p), p.cache.D) * 4;
}

cudaError_t launch_cache_attention(const CacheAttnProblem &p, int cache_dtype, cudaStream_t stream) {
    if (cache_dtype == FLEX_DTYPE_E4M3)
        return p.cache.D == 64 ? launch_cache_rows<64, true>(p, stream) : launch_cache_rows<128, true>(p, stream);
    return p.cache.D == 64 ? launch_cache_rows<64, false>(p, stream) : launch_cache_rows<128, false>(p, stream);
}

}  // namespace flex
