// Internal declarations of the attention over packed sequences: the plan's
// layout, and the problem handed from the C-ABI layer to the launchers.
#pragma once

#include "flex_internal.h"

namespace flex {

// A work item's Q tiles: two tiles of kBlock / G tokens of one sequence, G query
// heads of a token next to each other (row = token * G + head).
struct PlanEntry {
    int q_row;     // packed token of the first row
    int q_tokens;  // tokens of the sequence from there on
    int pos;       // position of the first token among the sequence's keys
    int k_row;     // packed token of the sequence's first key
    int k_len;
    int pad[3];
};
static_assert(sizeof(PlanEntry) == 32, "a plan's entries are read as two 16-byte words");

// The mask as plan and kernel see it; window INT32_MAX: every earlier token.
struct PackedMask {
    int causal, window, sinks;
};

struct PackedProblem {
    int sequences, Hq, Hk, D, total_q, total_k;
    const void *q, *k, *v;
    int64_t q_stride[2], k_stride[2], v_stride[2], out_stride[2];  // h, token (elements)
    const PlanEntry *plan;  // [0].q_row: how many entries follow
    int max_entries;
    PackedMask mask;
    int score_kind;
    float score_param, scale;
    uint16_t *out;
    float *lse;             // [Hq, total_q]
    int *status;
};

__host__ __device__ constexpr int packed_tile_tokens(int G) { return kBlock / G; }
__host__ __device__ constexpr int64_t packed_max_entries(int64_t total_q, int64_t sequences, int G) {
    return total_q / (2 * packed_tile_tokens(G)) + sequences;
}

// The kv tiles that a Q tile of positions first .. last needs: [lo, hi], and
// the first `sinks` tiles.
struct TileRange {
    int lo, hi, sinks;
};
__host__ __device__ __forceinline__ TileRange packed_range(const PackedMask &m, int first, int last, int k_len) {
    TileRange r = {0, -1, 0};
    if (!m.causal) {
        r.hi = (k_len - 1) >> 7;  // -1: no keys
    } else if (last >= 0 && k_len > 0) {
        const int64_t low = (int64_t)first - m.window + 1;
        r.lo = low > 0 ? (int)(low >> 7) : 0;
        r.hi = last >> 7;
        const int seen = m.sinks < last + 1 ? m.sinks : last + 1;
        r.sinks = (int)(((int64_t)seen + 127) >> 7);
    }
    return r;
}

// The kv tiles that all rows of positions first .. last keep whole: [lo, hi], and
// the first `sinks` tiles.
__host__ __device__ __forceinline__ TileRange packed_full(const PackedMask &m, int first, int last, int k_len) {
    TileRange r = {0, (k_len >> 7) - 1, 0};
    if (m.causal) {
        const int seen = first + 1 < k_len ? first + 1 : k_len;
        if (seen <= 0) return {0, -1, 0};
        const int64_t low = (int64_t)last - m.window + 1;
        r.lo = low > 0 ? (int)((low + 127) >> 7) : 0;
        r.hi = (seen >> 7) - 1;
        r.sinks = (m.sinks < seen ? m.sinks : seen) >> 7;
    }
    return r;
}

// The kv tiles of an item's two Q tiles together (`tokens` of them from position
// `pos` on, `per` a tile): hi, hi - 1, ... (n_main of them), then n_sink - 1, ... 0.
struct ItemTiles {
    TileRange range[2];
    int hi, n_main, n_sink;
};
__host__ __device__ __forceinline__ ItemTiles packed_item_tiles(const PackedMask &m, int pos, int tokens, int per, int k_len) {
    ItemTiles t;
    t.range[0] = packed_range(m, pos, pos + (tokens < per ? tokens : per) - 1, k_len);
    t.range[1] = {0, -1, 0};
    if (tokens > per) t.range[1] = packed_range(m, pos + per, pos + tokens - 1, k_len);
    int lo = t.range[0].lo;
    t.hi = t.range[0].hi;
    if (lo > t.hi) {
        lo = t.range[1].lo;
        t.hi = t.range[1].hi;
    } else if (t.range[1].lo <= t.range[1].hi) {  // neighbouring tokens: the ranges meet or overlap
        lo = lo < t.range[1].lo ? lo : t.range[1].lo;
        t.hi = t.hi > t.range[1].hi ? t.hi : t.range[1].hi;
    }
    t.n_main = t.hi - lo + 1 > 0 ? t.hi - lo + 1 : 0;
    const int sinks = t.range[0].sinks > t.range[1].sinks ? t.range[0].sinks : t.range[1].sinks;
    t.n_sink = t.n_main > 0 && lo < sinks ? lo : sinks;
    return t;
}

cudaError_t launch_packed_plan(const int32_t *q_starts, const int32_t *k_starts, int sequences, int total_q, int total_k,
                               int G, const PackedMask &mask, PlanEntry *plan, int max_entries, cudaStream_t stream);
cudaError_t launch_attn_packed(const PackedProblem &p, cudaStream_t stream);

}  // namespace flex
