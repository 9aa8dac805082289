// C-ABI layer of the attention over packed sequences (include/flexattn.h):
// argument checks on the host and dispatch to the kernels.
#include <climits>
#include <cmath>

#include "attn_packed.h"

namespace flex {
namespace {

bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

int check_heads(int32_t sequences, int32_t total_q, int32_t Hq, int32_t Hk) {
    if (sequences <= 0 || total_q <= 0 || Hq <= 0 || Hk <= 0 || Hq % Hk != 0) return FLEX_ERR_SHAPE;
    const int G = Hq / Hk;
    if (sequences > 65535 || Hq > 32767 || G > kBlock) return FLEX_ERR_UNSUPPORTED;
    return packed_max_entries(total_q, sequences, G) * Hk > INT_MAX ? FLEX_ERR_UNSUPPORTED : FLEX_OK;
}

int check_mask(int32_t kind, const flex_mask_params *params, PackedMask &mask) {
    mask = {kind != FLEX_MASK_ALL, INT_MAX, 0};
    switch (kind) {
        case FLEX_MASK_CAUSAL:
        case FLEX_MASK_ALL:
            return FLEX_OK;
        case FLEX_MASK_SLIDING_WINDOW:
        case FLEX_MASK_WINDOW_SINKS:
            if (!params || !valid_window(kind, *params)) return FLEX_ERR_INVALID_ARG;
            mask.window = params->window;
            mask.sinks = kind == FLEX_MASK_WINDOW_SINKS ? params->prefix : 0;
            return FLEX_OK;
        case FLEX_MASK_CAUSAL_PREFIX:
        case FLEX_MASK_DOCUMENT:
            return FLEX_ERR_UNSUPPORTED;
        default:
            return FLEX_ERR_INVALID_ARG;
    }
}

void take_strides(const flex_tensor *t, int64_t (&s)[2]) {
    s[0] = t->stride[1];
    s[1] = t->stride[2];
}

}  // namespace
}  // namespace flex

using namespace flex;

extern "C" {

int flex_packed_plan_bytes(int32_t sequences, int32_t total_q, int32_t Hq, int32_t Hk, int64_t *bytes) {
    if (!bytes) return FLEX_ERR_INVALID_ARG;
    const int rc = check_heads(sequences, total_q, Hq, Hk);
    if (rc == FLEX_OK) *bytes = (1 + packed_max_entries(total_q, sequences, Hq / Hk)) * (int64_t)sizeof(PlanEntry);
    return rc;
}

int flex_packed_plan_create(const int32_t *q_starts, const int32_t *k_starts, int32_t sequences, int32_t total_q,
                            int32_t total_k, int32_t Hq, int32_t Hk, int32_t mask_kind, const flex_mask_params *params,
                            flex_packed_plan *plan, void *stream) {
    if (!q_starts || !k_starts || !plan || !plan->entries) return FLEX_ERR_INVALID_ARG;
    int rc = check_heads(sequences, total_q, Hq, Hk);
    if (rc != FLEX_OK) return rc;
    if (total_k <= 0) return FLEX_ERR_SHAPE;
    PackedMask mask;
    if ((rc = check_mask(mask_kind, params, mask)) != FLEX_OK) return rc;
    if (!aligned(q_starts, 4) || !aligned(k_starts, 4) || !aligned(plan->entries, 16)) return FLEX_ERR_ALIGNMENT;
    plan->sequences = sequences;
    plan->total_q = total_q;
    plan->total_k = total_k;
    plan->Hq = Hq;
    plan->Hk = Hk;
    plan->mask_kind = mask_kind;
    plan->window = mask.window;
    plan->sinks = mask.sinks;
    return launch_packed_plan(q_starts, k_starts, sequences, total_q, total_k, Hq / Hk, mask,
                              static_cast<PlanEntry *>(plan->entries), (int)packed_max_entries(total_q, sequences, Hq / Hk),
                              static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FLEX_OK
               : FLEX_ERR_CUDA;
}

int flex_attention_packed_fwd(const flex_tensor *q, const flex_tensor *k, const flex_tensor *v, const flex_packed_plan *plan,
                              int32_t score_kind, float score_param, float scale, const flex_tensor *out, float *lse,
                              void *stream) {
    if (!q || !k || !v || !plan || !plan->entries || !out || !lse) return FLEX_ERR_INVALID_ARG;
    if (q->dtype != FLEX_DTYPE_BF16 && q->dtype != FLEX_DTYPE_FP32) return FLEX_ERR_INVALID_ARG;
    if (q->dtype != FLEX_DTYPE_BF16) return FLEX_ERR_UNSUPPORTED;
    if (score_kind < FLEX_SCORE_IDENTITY || score_kind > FLEX_SCORE_ALIBI) return FLEX_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return FLEX_ERR_INVALID_ARG;
    if (score_kind == FLEX_SCORE_SOFTCAP && !(score_param > 0.f && std::isfinite(score_param)))
        return FLEX_ERR_INVALID_ARG;
    int rc = check_heads(plan->sequences, plan->total_q, plan->Hq, plan->Hk);
    if (rc != FLEX_OK) return rc;
    const int64_t D = q->shape[3];
    if (D <= 0 || plan->total_k <= 0) return FLEX_ERR_SHAPE;
    if (D != 64 && D != 128) return FLEX_ERR_UNSUPPORTED;
    PackedProblem p = {};
    const flex_mask_params params = {plan->window, plan->sinks, nullptr};
    if ((rc = check_mask(plan->mask_kind, &params, p.mask)) != FLEX_OK) return rc;
    if ((rc = check_tensor(q, FLEX_DTYPE_BF16, 1, plan->Hq, plan->total_q, D)) != FLEX_OK) return rc;
    if ((rc = check_tensor(k, FLEX_DTYPE_BF16, 1, plan->Hk, plan->total_k, D)) != FLEX_OK) return rc;
    if ((rc = check_tensor(v, FLEX_DTYPE_BF16, 1, plan->Hk, plan->total_k, D)) != FLEX_OK) return rc;
    if ((rc = check_tensor(out, FLEX_DTYPE_BF16, 1, plan->Hq, plan->total_q, D)) != FLEX_OK) return rc;
    if (!aligned(lse, 4) || !aligned(plan->entries, 16)) return FLEX_ERR_ALIGNMENT;
    p.sequences = plan->sequences;
    p.Hq = plan->Hq;
    p.Hk = plan->Hk;
    p.D = (int)D;
    p.total_q = plan->total_q;
    p.total_k = plan->total_k;
    p.q = q->data;
    p.k = k->data;
    p.v = v->data;
    take_strides(q, p.q_stride);
    take_strides(k, p.k_stride);
    take_strides(v, p.v_stride);
    take_strides(out, p.out_stride);
    p.plan = static_cast<const PlanEntry *>(plan->entries);
    p.max_entries = (int)packed_max_entries(plan->total_q, plan->sequences, plan->Hq / plan->Hk);
    p.score_kind = score_kind;
    p.score_param = score_param;
    p.scale = scale;
    p.out = static_cast<uint16_t *>(const_cast<void *>(out->data));
    p.lse = lse;
    p.status = device_status_word(&rc);
    if (!p.status) return rc;
    return launch_attn_packed(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FLEX_OK : FLEX_ERR_CUDA;
}

}  // extern "C"
