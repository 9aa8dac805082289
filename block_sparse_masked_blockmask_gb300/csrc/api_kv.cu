// C-ABI layer of the rotary positions and the paged key/value cache
// (include/flexattn.h): argument checks on the host and dispatch to the
// kernels.  None of these calls synchronises, allocates (but the per-device
// status word of the attention, on its first call) or keeps state.
#include <climits>
#include <cmath>
#include <cstdint>

#include "kv_internal.h"

namespace flex {
namespace {

bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

constexpr int64_t kMaxCacheLen = int64_t(1) << 30;  // positions a page table may address

int check_rope(const flex_rope_params *r, int64_t D) {
    if (!r || !r->inv_freq) return FLEX_ERR_INVALID_ARG;
    if (r->layout != FLEX_ROPE_HALF && r->layout != FLEX_ROPE_INTERLEAVED) return FLEX_ERR_INVALID_ARG;
    if (!std::isfinite(r->attention_scale)) return FLEX_ERR_INVALID_ARG;
    if (r->rotary_dim <= 0 || r->rotary_dim > D) return FLEX_ERR_SHAPE;
    if (r->rotary_dim % 16 != 0) return FLEX_ERR_UNSUPPORTED;
    if (!aligned(r->inv_freq, 8)) return FLEX_ERR_ALIGNMENT;
    return FLEX_OK;
}

int check_dtype_dim(const flex_tensor *t) {
    if (!t) return FLEX_ERR_INVALID_ARG;
    if (t->dtype != FLEX_DTYPE_BF16 && t->dtype != FLEX_DTYPE_FP32) return FLEX_ERR_INVALID_ARG;
    if (t->shape[0] <= 0 || t->shape[1] <= 0 || t->shape[2] <= 0 || t->shape[3] <= 0) return FLEX_ERR_SHAPE;
    if (t->shape[3] != 64 && t->shape[3] != 128) return FLEX_ERR_UNSUPPORTED;
    if (t->shape[0] > 65535 || t->shape[1] > 32767 || t->shape[2] > INT32_MAX) return FLEX_ERR_UNSUPPORTED;
    return FLEX_OK;
}

void take_strides(const flex_tensor *t, int64_t (&s)[3]) {
    for (int i = 0; i < 3; ++i) s[i] = t->stride[i];
}

int rope(const flex_tensor *q, const flex_tensor *k, const flex_rope_params *r, const int32_t *positions,
         const flex_tensor *q_out, const flex_tensor *k_out, float direction, void *stream) {
    int rc = check_dtype_dim(q);
    if (rc != FLEX_OK) return rc;
    if (!q_out || (k != nullptr) != (k_out != nullptr)) return FLEX_ERR_INVALID_ARG;
    const int64_t B = q->shape[0], S = q->shape[2], D = q->shape[3];
    if ((rc = check_rope(r, D)) != FLEX_OK) return rc;
    if ((rc = check_tensor(q, q->dtype, B, q->shape[1], S, D)) != FLEX_OK) return rc;
    if ((rc = check_tensor(q_out, q->dtype, B, q->shape[1], S, D)) != FLEX_OK) return rc;
    if (k) {
        if ((rc = check_dtype_dim(k)) != FLEX_OK) return rc;
        if ((rc = check_tensor(k, q->dtype, B, k->shape[1], S, D)) != FLEX_OK) return rc;
        if ((rc = check_tensor(k_out, q->dtype, B, k->shape[1], S, D)) != FLEX_OK) return rc;
    }
    if (!aligned(positions, 4)) return FLEX_ERR_ALIGNMENT;
    if (B * S * (D / 8) > (int64_t)INT32_MAX * 128) return FLEX_ERR_UNSUPPORTED;  // CTAs along grid.x
    RopeProblem p = {};
    p.B = (int)B;
    p.S = (int)S;
    p.D = (int)D;
    const flex_tensor *in[2] = {q, k}, *out[2] = {q_out, k_out};
    for (int w = 0; w < (k ? 2 : 1); ++w) {
        p.heads[w] = (int)in[w]->shape[1];
        p.in[w] = in[w]->data;
        p.out[w] = const_cast<void *>(out[w]->data);
        take_strides(in[w], p.in_stride[w]);
        take_strides(out[w], p.out_stride[w]);
    }
    p.inv_freq = r->inv_freq;
    p.positions = positions;
    p.rotary = r->rotary_dim;
    p.layout = r->layout;
    p.attention_scale = r->attention_scale;
    p.direction = direction;
    return launch_rope(p, q->dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FLEX_OK : FLEX_ERR_CUDA;
}

int check_tables(const int32_t *page_table, const int32_t *lens) {
    if (!page_table || !lens) return FLEX_ERR_INVALID_ARG;
    return aligned(page_table, 4) && aligned(lens, 4) ? FLEX_OK : FLEX_ERR_ALIGNMENT;
}

int check_cache(const flex_kv_cache *c, int32_t max_pages) {
    if (!c || !c->k || !c->v) return FLEX_ERR_INVALID_ARG;
    if (c->dtype != FLEX_DTYPE_BF16 && c->dtype != FLEX_DTYPE_E4M3) return FLEX_ERR_INVALID_ARG;
    if (c->dtype == FLEX_DTYPE_E4M3 && (!c->k_scale || !c->v_scale)) return FLEX_ERR_INVALID_ARG;
    if (c->num_pages <= 0 || c->H <= 0 || c->page_size <= 0 || c->D <= 0 || max_pages <= 0) return FLEX_ERR_SHAPE;
    if (c->D != 64 && c->D != 128) return FLEX_ERR_UNSUPPORTED;
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return FLEX_ERR_UNSUPPORTED;
    if (c->H > 32767 || (int64_t)c->num_pages * c->H > INT32_MAX || (int64_t)max_pages * c->page_size > kMaxCacheLen) return FLEX_ERR_UNSUPPORTED;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return FLEX_ERR_ALIGNMENT;
    return FLEX_OK;
}

KvCache cache_of(const flex_kv_cache *c) {
    int shift = 4;
    while ((1 << shift) < c->page_size) ++shift;
    return KvCache{c->num_pages, c->H, c->page_size, c->D, shift, static_cast<uint8_t *>(c->k),
                   static_cast<uint8_t *>(c->v), c->k_scale, c->v_scale};
}

// The checks of sizes, types and mask that the attention and its workspace
// share; on success p holds what they describe.
int cache_problem(const flex_tensor *q, const flex_kv_cache *cache, int32_t max_pages, int32_t mask_kind,
                  const flex_mask_params *params, CacheAttnProblem &p) {
    int rc = check_cache(cache, max_pages);
    if (rc == FLEX_OK) rc = check_dtype_dim(q);
    if (rc != FLEX_OK) return rc;
    if (q->dtype != FLEX_DTYPE_BF16) return FLEX_ERR_UNSUPPORTED;
    switch (mask_kind) {
        case FLEX_MASK_CAUSAL:
        case FLEX_MASK_ALL:
            break;
        case FLEX_MASK_SLIDING_WINDOW:
        case FLEX_MASK_WINDOW_SINKS:
            if (!params || !valid_window(mask_kind, *params)) return FLEX_ERR_INVALID_ARG;
            break;
        case FLEX_MASK_CAUSAL_PREFIX:
        case FLEX_MASK_DOCUMENT:
            return FLEX_ERR_UNSUPPORTED;
        default:
            return FLEX_ERR_INVALID_ARG;
    }
    if (q->shape[3] != cache->D || q->shape[1] % cache->H != 0) return FLEX_ERR_SHAPE;
    if ((rc = check_tensor(q, FLEX_DTYPE_BF16, q->shape[0], q->shape[1], q->shape[2], cache->D)) != FLEX_OK) return rc;
    p.B = (int)q->shape[0];
    p.Hq = (int)q->shape[1];
    p.G = p.Hq / cache->H;
    p.Q = (int)q->shape[2];
    // (sequence, head, row tile) triples along grid.x
    if ((int64_t)p.Q * p.G > kMaxCacheLen || (int64_t)p.B * cache->H * (((int64_t)p.Q * p.G + 7) / 8) > INT32_MAX)
        return FLEX_ERR_UNSUPPORTED;
    p.cache = cache_of(cache);
    p.max_pages = max_pages;
    const bool windowed = mask_kind == FLEX_MASK_SLIDING_WINDOW || mask_kind == FLEX_MASK_WINDOW_SINKS;
    p.window = windowed ? params->window : INT_MAX;
    p.sinks = mask_kind == FLEX_MASK_WINDOW_SINKS ? params->prefix : 0;
    p.causal = mask_kind != FLEX_MASK_ALL;
    return FLEX_OK;
}

}  // namespace
}  // namespace flex

using namespace flex;

extern "C" {

int flex_rope_frequencies(int32_t rotary_dim, double base, int32_t scaling, double factor, double original_len,
                          double low_turns, double high_turns, double *inv_freq) {
    if (!inv_freq || rotary_dim <= 0 || rotary_dim % 2 != 0) return FLEX_ERR_INVALID_ARG;
    if (!(base > 0) || !std::isfinite(base)) return FLEX_ERR_INVALID_ARG;
    if (scaling < FLEX_ROPE_SCALE_NONE || scaling > FLEX_ROPE_SCALE_PARTS) return FLEX_ERR_INVALID_ARG;
    if (scaling != FLEX_ROPE_SCALE_NONE && !(factor >= 1 && std::isfinite(factor))) return FLEX_ERR_INVALID_ARG;
    if (scaling == FLEX_ROPE_SCALE_PARTS && !(original_len > 0 && std::isfinite(original_len) && low_turns >= 0 &&
                                              high_turns > low_turns && std::isfinite(high_turns)))
        return FLEX_ERR_INVALID_ARG;
    if (scaling == FLEX_ROPE_SCALE_BASE) {
        if (rotary_dim == 2) return FLEX_ERR_INVALID_ARG;
        base *= std::pow(factor, (double)rotary_dim / (rotary_dim - 2));
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rotary_dim);
        if (scaling == FLEX_ROPE_SCALE_LINEAR) f /= factor;
        if (scaling == FLEX_ROPE_SCALE_PARTS) {
            const double turns = original_len * f / 6.283185307179586477;
            double keep = (turns - low_turns) / (high_turns - low_turns);
            keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
            f *= keep + (1 - keep) / factor;
        }
        inv_freq[i] = f;
    }
    return FLEX_OK;
}

int flex_rope_fwd(const flex_tensor *q, const flex_tensor *k, const flex_rope_params *r, const int32_t *positions,
                  const flex_tensor *q_out, const flex_tensor *k_out, void *stream) {
    return rope(q, k, r, positions, q_out, k_out, 1.f, stream);
}

int flex_rope_bwd(const flex_tensor *dq, const flex_tensor *dk, const flex_rope_params *r, const int32_t *positions,
                  const flex_tensor *dq_out, const flex_tensor *dk_out, void *stream) {
    return rope(dq, dk, r, positions, dq_out, dk_out, -1.f, stream);
}

int flex_kv_cache_append(const flex_kv_cache *cache, const flex_tensor *k, const flex_tensor *v,
                         const int32_t *page_table, int32_t max_pages, const int32_t *cache_lens,
                         const int32_t *new_lens, const flex_rope_params *r, void *stream) {
    int rc = check_cache(cache, max_pages);
    if (rc == FLEX_OK) rc = check_tables(page_table, cache_lens);
    if (rc != FLEX_OK) return rc;
    if ((rc = check_dtype_dim(k)) != FLEX_OK) return rc;
    if (k->shape[3] != cache->D || k->shape[1] != cache->H) return FLEX_ERR_SHAPE;
    if ((rc = check_tensor(k, k->dtype, k->shape[0], cache->H, k->shape[2], cache->D)) != FLEX_OK) return rc;
    if ((rc = check_tensor(v, k->dtype, k->shape[0], cache->H, k->shape[2], cache->D)) != FLEX_OK) return rc;
    if (r && (rc = check_rope(r, cache->D)) != FLEX_OK) return rc;
    if (!aligned(new_lens, 4)) return FLEX_ERR_ALIGNMENT;
    AppendProblem p = {};
    p.B = (int)k->shape[0];
    p.S = (int)k->shape[2];
    p.cache = cache_of(cache);
    p.k = k->data;
    p.v = v->data;
    take_strides(k, p.k_stride);
    take_strides(v, p.v_stride);
    p.page_table = page_table;
    p.max_pages = max_pages;
    p.cache_lens = cache_lens;
    p.new_lens = new_lens;
    if (r) {
        p.inv_freq = r->inv_freq;
        p.rotary = r->rotary_dim;
        p.layout = r->layout;
        p.attention_scale = r->attention_scale;
    }
    return launch_kv_append(p, k->dtype, cache->dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FLEX_OK
               : FLEX_ERR_CUDA;
}

int flex_kv_cache_attention_workspace(const flex_tensor *q, const flex_kv_cache *cache, int32_t max_pages,
                                      int32_t mask_kind, const flex_mask_params *params, int64_t *bytes) {
    if (!bytes) return FLEX_ERR_INVALID_ARG;
    CacheAttnProblem p = {};
    const int rc = cache_problem(q, cache, max_pages, mask_kind, params, p);
    if (rc != FLEX_OK) return rc;
    *bytes = cache_attention_workspace(p, cache->dtype);
    return FLEX_OK;
}

int flex_kv_cache_attention(const flex_tensor *q, const flex_kv_cache *cache, const int32_t *page_table,
                            int32_t max_pages, const int32_t *kv_lens, int32_t mask_kind,
                            const flex_mask_params *params, int32_t score_kind, float score_param, float scale,
                            void *out, float *lse, void *workspace, int64_t workspace_bytes, void *stream) {
    CacheAttnProblem p = {};
    int rc = cache_problem(q, cache, max_pages, mask_kind, params, p);
    if (rc == FLEX_OK) rc = check_tables(page_table, kv_lens);
    if (rc != FLEX_OK) return rc;
    if (!out || !lse || !workspace) return FLEX_ERR_INVALID_ARG;
    if (score_kind < FLEX_SCORE_IDENTITY || score_kind > FLEX_SCORE_ALIBI) return FLEX_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return FLEX_ERR_INVALID_ARG;
    if (score_kind == FLEX_SCORE_SOFTCAP && !(score_param > 0.f && std::isfinite(score_param)))
        return FLEX_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16)) return FLEX_ERR_ALIGNMENT;
    if (workspace_bytes < cache_attention_workspace(p, cache->dtype)) return FLEX_ERR_SHAPE;
    p.q = static_cast<const uint16_t *>(q->data);
    take_strides(q, p.q_stride);
    p.page_table = page_table;
    p.kv_lens = kv_lens;
    p.score_kind = score_kind;
    p.score_param = score_param;
    p.scale = scale;
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.workspace = workspace;
    p.status = device_status_word(&rc);
    if (!p.status) return rc;
    return launch_cache_attention(p, cache->dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FLEX_OK
                                                                                                     : FLEX_ERR_CUDA;
}

}  // extern "C"
