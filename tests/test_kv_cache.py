"""Rotary positions and the paged cache: what the host refuses (no GPU needed;
every call fails its checks before any CUDA call)."""
import ctypes
import math

import pytest
import torch

from block_sparse_masked_blockmask_gb300 import _build, flexattn as fa
from test_abi import _tensor

BF, F32, E4 = fa.FLEX_DTYPE_BF16, fa.FLEX_DTYPE_FP32, fa.FLEX_DTYPE_E4M3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load_library()


def changed(struct, **fields):
    out = type(struct).from_buffer_copy(struct)
    for k, v in fields.items():
        setattr(out, k, v)
    return out


ROPE = fa.flex_rope_params(0x1000, 64, fa.FLEX_ROPE_HALF, 1.0, 0)
CACHE = fa.flex_kv_cache(10, 2, 64, 128, E4, 0, 0x1000, 0x2000, 0x3000, 0x4000)


def ref(x):
    return None if x is None else ctypes.byref(x)


BAD_ROPE = [
    (dict(inv_freq=None), fa.FLEX_ERR_INVALID_ARG),
    (dict(layout=2), fa.FLEX_ERR_INVALID_ARG),
    (dict(attention_scale=math.inf), fa.FLEX_ERR_INVALID_ARG),
    (dict(rotary_dim=0), fa.FLEX_ERR_SHAPE),
    (dict(rotary_dim=144), fa.FLEX_ERR_SHAPE),
    (dict(rotary_dim=24), fa.FLEX_ERR_UNSUPPORTED),
    (dict(inv_freq=0x1004), fa.FLEX_ERR_ALIGNMENT),
]


@pytest.mark.parametrize("name", ["flex_rope_fwd", "flex_rope_bwd"])
def test_rope_refusals(lib, name):
    q, k = _tensor(BF, [2, 4, 8, 128]), _tensor(BF, [2, 2, 8, 128])

    def call(q=q, k=k, r=ROPE, positions=0x2000, q_out=q, k_out=k):
        return getattr(lib, name)(ref(q), ref(k), ref(r), positions, ref(q_out), ref(k_out), None)

    for fields, code in BAD_ROPE:
        assert call(r=changed(ROPE, **fields)) == code, fields
    assert call(q=None) == fa.FLEX_ERR_INVALID_ARG
    assert call(r=None) == fa.FLEX_ERR_INVALID_ARG
    assert call(k=None) == fa.FLEX_ERR_INVALID_ARG        # an output for nothing
    assert call(k_out=None) == fa.FLEX_ERR_INVALID_ARG
    assert call(positions=0x2002) == fa.FLEX_ERR_ALIGNMENT
    assert call(q_out=_tensor(F32, [2, 4, 8, 128])) == fa.FLEX_ERR_INVALID_ARG
    assert call(k=_tensor(F32, [2, 2, 8, 128])) == fa.FLEX_ERR_INVALID_ARG
    assert call(q=_tensor(E4, [2, 4, 8, 128])) == fa.FLEX_ERR_INVALID_ARG
    assert call(k=_tensor(BF, [2, 2, 9, 128])) == fa.FLEX_ERR_SHAPE
    assert call(q_out=_tensor(BF, [2, 4, 8, 64])) == fa.FLEX_ERR_SHAPE
    assert call(q=_tensor(BF, [2, 4, 8, 96])) == fa.FLEX_ERR_UNSUPPORTED
    assert call(q=_tensor(BF, [2, 4, 0, 128])) == fa.FLEX_ERR_SHAPE
    assert call(q=_tensor(BF, [2, 4, 8, 128], stride=[4096, 0, 128, 1])) == fa.FLEX_ERR_ALIGNMENT
    assert call(q_out=_tensor(BF, [2, 4, 8, 128], stride=[4096, 1024, 132, 1])) == fa.FLEX_ERR_ALIGNMENT
    assert call(q=_tensor(BF, [2, 4, 8, 128], data=0x10008)) == fa.FLEX_ERR_ALIGNMENT
    assert call(q=_tensor(BF, [70000, 4, 8, 128])) == fa.FLEX_ERR_UNSUPPORTED


def test_frequency_refusals(lib):
    for args in ((0,), (7,), (64, 0.0), (64, math.inf), (64, 1e4, 4), (64, 1e4, 1, 0.5), (64, 1e4, 3, 2.0, 0.0),
                 (64, 1e4, 3, 2.0, 100.0, 4.0, 4.0), (64, 1e4, 3, 2.0, 100.0, -1.0, 4.0), (2, 1e4, 2, 2.0)):
        with pytest.raises(fa.FlexError) as e:
            fa.flex_rope_frequencies(*args, device="cpu")
        assert e.value.code == fa.FLEX_ERR_INVALID_ARG, args


BAD_CACHE = [
    (dict(k=None), fa.FLEX_ERR_INVALID_ARG),
    (dict(v=None), fa.FLEX_ERR_INVALID_ARG),
    (dict(k_scale=None), fa.FLEX_ERR_INVALID_ARG),
    (dict(dtype=F32), fa.FLEX_ERR_INVALID_ARG),
    (dict(num_pages=0), fa.FLEX_ERR_SHAPE),
    (dict(H=0), fa.FLEX_ERR_SHAPE),
    (dict(D=96), fa.FLEX_ERR_UNSUPPORTED),
    (dict(page_size=8), fa.FLEX_ERR_UNSUPPORTED),
    (dict(page_size=48), fa.FLEX_ERR_UNSUPPORTED),
    (dict(page_size=512), fa.FLEX_ERR_UNSUPPORTED),
    (dict(v=0x2008), fa.FLEX_ERR_ALIGNMENT),
    (dict(v_scale=0x4002), fa.FLEX_ERR_ALIGNMENT),
]


def test_append_refusals(lib):
    k = _tensor(BF, [3, 2, 5, 128])

    def call(cache=CACHE, k=k, v=k, table=0x5000, width=4, lens=0x6000, new=None, rope=ROPE):
        return lib.flex_kv_cache_append(ref(cache), ref(k), ref(v), table, width, lens, new, ref(rope), None)

    for fields, code in BAD_CACHE:
        assert call(cache=changed(CACHE, **fields)) == code, fields
    for fields, code in BAD_ROPE:
        assert call(rope=changed(ROPE, **fields)) == code, fields
    assert call(cache=None) == fa.FLEX_ERR_INVALID_ARG
    assert call(table=None) == fa.FLEX_ERR_INVALID_ARG
    assert call(lens=None) == fa.FLEX_ERR_INVALID_ARG
    assert call(width=0) == fa.FLEX_ERR_SHAPE
    assert call(width=2**25) == fa.FLEX_ERR_UNSUPPORTED
    assert call(table=0x5002) == fa.FLEX_ERR_ALIGNMENT
    assert call(new=0x6002) == fa.FLEX_ERR_ALIGNMENT
    assert call(k=None) == fa.FLEX_ERR_INVALID_ARG
    assert call(v=_tensor(BF, [3, 2, 6, 128])) == fa.FLEX_ERR_SHAPE
    assert call(v=_tensor(F32, [3, 2, 5, 128])) == fa.FLEX_ERR_INVALID_ARG
    assert call(k=_tensor(BF, [3, 4, 5, 128])) == fa.FLEX_ERR_SHAPE
    assert call(k=_tensor(BF, [3, 2, 5, 64])) == fa.FLEX_ERR_SHAPE


def test_attention_refusals(lib):
    q = _tensor(BF, [3, 6, 1, 128])
    good = fa.flex_mask_params(4, 1, None)

    def call(q=q, cache=CACHE, table=0x5000, width=4, lens=0x6000, kind=fa.FLEX_MASK_CAUSAL, params=good,
             score=fa.FLEX_SCORE_IDENTITY, param=0.0, scale=0.1, out=0x7000, lse=0x8000, work=0x9000, size=1 << 24):
        return lib.flex_kv_cache_attention(ref(q), ref(cache), table, width, lens, kind, ref(params), score, param,
                                           scale, out, lse, work, size, None)

    for fields, code in BAD_CACHE:
        assert call(cache=changed(CACHE, **fields)) == code, fields
    assert call(q=_tensor(F32, [3, 6, 1, 128])) == fa.FLEX_ERR_UNSUPPORTED
    assert call(q=_tensor(BF, [3, 5, 1, 128])) == fa.FLEX_ERR_SHAPE
    assert call(q=_tensor(BF, [3, 6, 1, 64])) == fa.FLEX_ERR_SHAPE
    assert call(q=_tensor(BF, [3, 6, 0, 128])) == fa.FLEX_ERR_SHAPE
    assert call(q=None) == fa.FLEX_ERR_INVALID_ARG
    assert call(out=None) == fa.FLEX_ERR_INVALID_ARG
    assert call(lse=None) == fa.FLEX_ERR_INVALID_ARG
    assert call(out=0x7008) == fa.FLEX_ERR_ALIGNMENT
    assert call(lse=0x8002) == fa.FLEX_ERR_ALIGNMENT
    assert call(kind=fa.FLEX_MASK_DOCUMENT) == fa.FLEX_ERR_UNSUPPORTED
    assert call(kind=fa.FLEX_MASK_CAUSAL_PREFIX) == fa.FLEX_ERR_UNSUPPORTED
    assert call(kind=6) == fa.FLEX_ERR_INVALID_ARG
    for kind in (fa.FLEX_MASK_SLIDING_WINDOW, fa.FLEX_MASK_WINDOW_SINKS):
        assert call(kind=kind, params=None) == fa.FLEX_ERR_INVALID_ARG
        assert call(kind=kind, params=fa.flex_mask_params(-1, 0, None)) == fa.FLEX_ERR_INVALID_ARG
    assert call(kind=fa.FLEX_MASK_WINDOW_SINKS, params=fa.flex_mask_params(1, -1, None)) == fa.FLEX_ERR_INVALID_ARG
    assert call(score=3) == fa.FLEX_ERR_INVALID_ARG
    assert call(score=fa.FLEX_SCORE_SOFTCAP) == fa.FLEX_ERR_INVALID_ARG
    assert call(scale=math.nan) == fa.FLEX_ERR_INVALID_ARG
    assert call(table=None) == fa.FLEX_ERR_INVALID_ARG
    assert call(lens=0x6002) == fa.FLEX_ERR_ALIGNMENT
    assert call(work=None) == fa.FLEX_ERR_INVALID_ARG
    assert call(work=0x9008) == fa.FLEX_ERR_ALIGNMENT
    size = ctypes.c_int64()
    need = lambda q=q, cache=CACHE, kind=fa.FLEX_MASK_CAUSAL: lib.flex_kv_cache_attention_workspace(  # noqa: E731
        ref(q), ref(cache), 4, kind, ref(good), ctypes.byref(size))
    assert need() == fa.FLEX_OK and 0 < size.value <= 4 << 20
    assert call(size=size.value - 1) == fa.FLEX_ERR_SHAPE
    assert need(q=_tensor(BF, [3, 5, 1, 128])) == fa.FLEX_ERR_SHAPE
    assert need(kind=fa.FLEX_MASK_DOCUMENT) == fa.FLEX_ERR_UNSUPPORTED
    assert need(q=_tensor(BF, [60000, 6, 1 << 20, 128])) == fa.FLEX_ERR_UNSUPPORTED
    assert lib.flex_kv_cache_attention_workspace(ref(q), ref(CACHE), 4, 0, None, None) == fa.FLEX_ERR_INVALID_ARG


def test_python_refusals(lib):
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    c = fa.KVCache(k, k.clone())
    with pytest.raises(ValueError):
        fa.KVCache(k, k[:3])
    with pytest.raises(ValueError):
        fa.KVCache(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn))
    with pytest.raises(ValueError):
        fa.KVCache(k, k, torch.zeros(4, 2), torch.zeros(4, 2))
    q = torch.zeros((3, 2, 1, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((3, 2), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for bad in (dict(page_table=table.long()), dict(page_table=table[:2]), dict(kv_lens=lens[:2]),
                dict(page_table=torch.zeros((3, 4), dtype=torch.int32)[:, ::2]), dict(kv_lens=lens.long()),
                dict(sinks=2), dict(out=q.float()), dict(lse=torch.zeros(3, 2))):
        with pytest.raises(ValueError):
            fa.flex_kv_cache_attention(**{**dict(q=q, cache=c, page_table=table, kv_lens=lens), **bad})
    with pytest.raises(ValueError):
        fa.flex_kv_cache_append(c, q, q, table, lens, lens.long())
    with pytest.raises(ValueError):
        fa.flex_kv_cache_append(c, q, q, table, lens, inv_freq=torch.zeros(16))
