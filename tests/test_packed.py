"""Attention over packed sequences: what the host refuses (no GPU needed; every call fails its checks before any CUDA
call)."""
import ctypes
import math

import pytest
import torch

from block_sparse_masked_blockmask_gb300 import _build, flexattn as fa
from test_abi import _tensor
from test_kv_cache import changed, ref

BF, F32 = fa.FLEX_DTYPE_BF16, fa.FLEX_DTYPE_FP32
PLAN = fa.flex_packed_plan(3, 50, 70, 8, 2, fa.FLEX_MASK_CAUSAL, 2**31 - 1, 0, 0x9000)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load_library()


def test_plan_bytes(lib):
    # runs of two tiles of 128 / G tokens, one more for every sequence, and the head
    assert fa.flex_packed_plan_bytes(3, 1000, 8, 8) == 32 * (1 + 1000 // 256 + 3)
    assert fa.flex_packed_plan_bytes(1, 1000, 8, 2) == 32 * (1 + 1000 // 64 + 1)
    assert fa.flex_packed_plan_bytes(2, 1000, 10, 2) == 32 * (1 + 1000 // 50 + 2)
    assert fa.flex_packed_plan_bytes(1, 7, 128, 1) == 32 * (1 + 3 + 1)
    for args, code in [((0, 10, 8, 2), fa.FLEX_ERR_SHAPE), ((1, 0, 8, 2), fa.FLEX_ERR_SHAPE), ((1, 10, 8, 3), fa.FLEX_ERR_SHAPE),
                       ((1, 10, 0, 1), fa.FLEX_ERR_SHAPE), ((1, 10, 8, 0), fa.FLEX_ERR_SHAPE),
                       ((70000, 10, 8, 2), fa.FLEX_ERR_UNSUPPORTED), ((1, 10, 129, 1), fa.FLEX_ERR_UNSUPPORTED),
                       ((1, 10, 40000, 40000), fa.FLEX_ERR_UNSUPPORTED), ((1, 2**31 - 1, 32000, 2000), fa.FLEX_ERR_UNSUPPORTED)]:
        with pytest.raises(fa.FlexError) as e:
            fa.flex_packed_plan_bytes(*args)
        assert e.value.code == code, args
    assert lib.flex_packed_plan_bytes(1, 10, 8, 2, None) == fa.FLEX_ERR_INVALID_ARG


def test_plan_refusals(lib):
    params = fa.flex_mask_params(4, 1, None)

    def call(qs=0x1000, ks=0x2000, n=3, tq=50, tk=70, Hq=8, Hk=2, kind=fa.FLEX_MASK_CAUSAL, params=params, plan=PLAN):
        return lib.flex_packed_plan_create(qs, ks, n, tq, tk, Hq, Hk, kind, ref(params), ref(plan), None)

    for missing in ("qs", "ks", "plan"):
        assert call(**{missing: None}) == fa.FLEX_ERR_INVALID_ARG, missing
    assert call(plan=changed(PLAN, entries=None)) == fa.FLEX_ERR_INVALID_ARG
    assert call(plan=changed(PLAN, entries=0x9008)) == fa.FLEX_ERR_ALIGNMENT
    assert call(qs=0x1002) == fa.FLEX_ERR_ALIGNMENT
    assert call(ks=0x2001) == fa.FLEX_ERR_ALIGNMENT
    assert call(n=0) == fa.FLEX_ERR_SHAPE
    assert call(tq=0) == fa.FLEX_ERR_SHAPE
    assert call(tk=0) == fa.FLEX_ERR_SHAPE
    assert call(Hq=7) == fa.FLEX_ERR_SHAPE
    assert call(Hq=258) == fa.FLEX_ERR_UNSUPPORTED
    assert call(n=65536) == fa.FLEX_ERR_UNSUPPORTED
    assert call(kind=fa.FLEX_MASK_DOCUMENT) == fa.FLEX_ERR_UNSUPPORTED
    assert call(kind=fa.FLEX_MASK_CAUSAL_PREFIX) == fa.FLEX_ERR_UNSUPPORTED
    assert call(kind=6) == fa.FLEX_ERR_INVALID_ARG
    for kind in (fa.FLEX_MASK_SLIDING_WINDOW, fa.FLEX_MASK_WINDOW_SINKS):
        assert call(kind=kind, params=None) == fa.FLEX_ERR_INVALID_ARG
        assert call(kind=kind, params=fa.flex_mask_params(-1, 0, None)) == fa.FLEX_ERR_INVALID_ARG
    assert call(kind=fa.FLEX_MASK_WINDOW_SINKS, params=fa.flex_mask_params(1, -1, None)) == fa.FLEX_ERR_INVALID_ARG


def test_attention_refusals(lib):
    q, k = _tensor(BF, [1, 8, 50, 128]), _tensor(BF, [1, 2, 70, 128])

    def call(q=q, k=k, v=k, plan=PLAN, score=fa.FLEX_SCORE_IDENTITY, param=0.0, scale=0.1, out=q, lse=0x8000):
        return lib.flex_attention_packed_fwd(ref(q), ref(k), ref(v), ref(plan), score, param, scale, ref(out), lse, None)

    for missing in ("q", "k", "v", "plan", "out", "lse"):
        assert call(**{missing: None}) == fa.FLEX_ERR_INVALID_ARG, missing
    f = _tensor(F32, [1, 8, 50, 128])
    assert call(q=f) == fa.FLEX_ERR_UNSUPPORTED
    assert call(k=_tensor(F32, [1, 2, 70, 128])) == fa.FLEX_ERR_INVALID_ARG
    assert call(out=f) == fa.FLEX_ERR_INVALID_ARG
    assert call(score=3) == fa.FLEX_ERR_INVALID_ARG
    assert call(score=fa.FLEX_SCORE_SOFTCAP) == fa.FLEX_ERR_INVALID_ARG
    assert call(score=fa.FLEX_SCORE_SOFTCAP, param=math.inf) == fa.FLEX_ERR_INVALID_ARG
    assert call(scale=math.nan) == fa.FLEX_ERR_INVALID_ARG
    assert call(lse=0x8002) == fa.FLEX_ERR_ALIGNMENT
    for bad in ([2, 8, 50, 128], [1, 4, 50, 128], [1, 8, 49, 128], [1, 8, 50, 64]):
        t = _tensor(BF, bad)
        assert call(out=t) == fa.FLEX_ERR_SHAPE, bad
        if bad[3] == 128:
            assert call(q=t, out=t) == fa.FLEX_ERR_SHAPE, bad
    for bad in ([1, 8, 70, 128], [1, 2, 71, 128], [1, 2, 70, 64], [2, 2, 70, 128]):
        assert call(v=_tensor(BF, bad)) == fa.FLEX_ERR_SHAPE, bad
    q96 = _tensor(BF, [1, 8, 50, 96])
    assert call(q=q96, out=q96) == fa.FLEX_ERR_UNSUPPORTED
    assert call(q=_tensor(BF, [1, 8, 50, 128], data=0x10008)) == fa.FLEX_ERR_ALIGNMENT
    assert call(out=_tensor(BF, [1, 8, 50, 128], stride=[51200, 6400, 132, 1])) == fa.FLEX_ERR_ALIGNMENT
    for fields, code in [(dict(entries=None), fa.FLEX_ERR_INVALID_ARG), (dict(entries=0x9004), fa.FLEX_ERR_ALIGNMENT),
                         (dict(mask_kind=fa.FLEX_MASK_DOCUMENT), fa.FLEX_ERR_UNSUPPORTED), (dict(Hk=3), fa.FLEX_ERR_SHAPE),
                         (dict(mask_kind=fa.FLEX_MASK_WINDOW_SINKS, sinks=-1), fa.FLEX_ERR_INVALID_ARG),
                         (dict(sequences=0), fa.FLEX_ERR_SHAPE), (dict(total_q=51), fa.FLEX_ERR_SHAPE),
                         (dict(total_k=69), fa.FLEX_ERR_SHAPE)]:
        assert call(plan=changed(PLAN, **fields)) == code, fields


def test_python_refusals(lib):
    starts = torch.tensor([0, 20, 50], dtype=torch.int32)
    good = dict(q_starts=starts, k_starts=starts, total_q=50, total_k=50, Hq=8, Hk=2)
    for bad in (dict(q_starts=starts.long()), dict(q_starts=starts[:1]), dict(k_starts=starts[:2]), dict(k_starts=starts.float()),
                dict(k_starts=None, total_k=60), dict(total_k=None), dict(sinks=2)):
        with pytest.raises(ValueError):
            fa.flex_packed_plan_create(**{**good, **bad})
    plan = fa.PackedPlan(changed(PLAN, total_k=50), torch.zeros(64, dtype=torch.uint8))
    q, k = torch.zeros((1, 8, 50, 64), dtype=torch.bfloat16), torch.zeros((1, 2, 50, 64), dtype=torch.bfloat16)
    good = dict(q=q, k=k, v=k, plan=plan)
    for bad in (dict(q=q[0]), dict(k=k.half()), dict(out=q.half()), dict(lse=torch.zeros(1, 8, 49)),
                dict(lse=torch.zeros((1, 8, 50), dtype=torch.float64)), dict(lse=torch.zeros(1, 50, 8).transpose(1, 2))):
        with pytest.raises(ValueError):
            fa.flex_attention_packed_fwd(**{**good, **bad})


def test_structure():
    assert fa.flex_packed_plan.entries.offset == 32 and ctypes.sizeof(fa.flex_packed_plan) == 40
