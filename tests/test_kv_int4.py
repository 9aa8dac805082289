"""The 4-bit cache, packed appends and the read: what the host refuses (no GPU needed; every call fails its
checks before any CUDA call)."""
import ctypes

import pytest
import torch

from block_sparse_masked_blockmask_gb300 import _build, flexattn as fa
from test_abi import _tensor
from test_kv_cache import BAD_CACHE, BAD_ROPE, ROPE, changed, ref

BF, F32, E4, I4 = fa.FLEX_DTYPE_BF16, fa.FLEX_DTYPE_FP32, fa.FLEX_DTYPE_E4M3, fa.FLEX_DTYPE_INT4
CACHE = fa.flex_kv_cache(10, 2, 64, 128, I4, 0, 0x1000, 0x2000, 0x3000, 0x4000)
BAD = BAD_CACHE + [(dict(v_scale=None), fa.FLEX_ERR_INVALID_ARG), (dict(k_scale=0x3004), fa.FLEX_ERR_ALIGNMENT),
                   (dict(v_scale=0x4008), fa.FLEX_ERR_ALIGNMENT), (dict(dtype=4), fa.FLEX_ERR_INVALID_ARG)]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load_library()


def test_append_refusals(lib):
    k = _tensor(BF, [3, 2, 5, 128])
    for fields, code in BAD:
        assert lib.flex_kv_cache_append(ref(changed(CACHE, **fields)), ref(k), ref(k), 0x5000, 4, 0x6000, None, None,
                                        None) == code, fields
    assert lib.flex_kv_cache_append(ref(CACHE), ref(k), ref(k), 0x5000, 4, 0x6000, 0x7001, None,
                                    None) == fa.FLEX_ERR_ALIGNMENT


@pytest.mark.parametrize("dtype", [BF, E4, I4])
def test_append_packed_refusals(lib, dtype):
    cache, k = changed(CACHE, dtype=dtype), _tensor(BF, [1, 2, 5, 128])

    def call(cache=cache, k=k, v=k, starts=0x8000, n=3, table=0x5000, width=4, lens=0x6000, rope=ROPE):
        return lib.flex_kv_cache_append_packed(ref(cache), ref(k), ref(v), starts, n, table, width, lens, ref(rope), None)

    for fields, code in BAD:
        if dtype == I4 or not any("scale" in f for f in fields):
            assert call(cache=changed(cache, **fields)) == code, fields
    for fields, code in BAD_ROPE:
        assert call(rope=changed(ROPE, **fields)) == code, fields
    for missing in ("cache", "k", "v", "starts", "table", "lens"):
        assert call(**{missing: None}) == fa.FLEX_ERR_INVALID_ARG, missing
    assert call(starts=0x8002) == fa.FLEX_ERR_ALIGNMENT
    assert call(n=0) == fa.FLEX_ERR_SHAPE
    assert call(n=-1) == fa.FLEX_ERR_SHAPE
    assert call(n=70000) == fa.FLEX_ERR_UNSUPPORTED
    assert call(width=0) == fa.FLEX_ERR_SHAPE
    two = _tensor(BF, [2, 2, 5, 128])
    assert call(k=two, v=two) == fa.FLEX_ERR_SHAPE          # packed tokens are one batch entry
    assert call(v=_tensor(BF, [1, 2, 6, 128])) == fa.FLEX_ERR_SHAPE
    assert call(v=_tensor(F32, [1, 2, 5, 128])) == fa.FLEX_ERR_INVALID_ARG
    assert call(k=_tensor(BF, [1, 3, 5, 128])) == fa.FLEX_ERR_SHAPE


@pytest.mark.parametrize("dtype", [BF, E4, I4])
def test_read_refusals(lib, dtype):
    cache, k = changed(CACHE, dtype=dtype), _tensor(BF, [1, 2, 5, 128])

    def call(cache=cache, k=k, v=k, starts=0x8000, n=3, table=0x5000, width=4):
        return lib.flex_kv_cache_read(ref(cache), table, width, starts, n, ref(k), ref(v), None)

    for fields, code in BAD:
        if dtype == I4 or not any("scale" in f for f in fields):
            assert call(cache=changed(cache, **fields)) == code, fields
    for missing in ("cache", "k", "v", "starts", "table"):
        assert call(**{missing: None}) == fa.FLEX_ERR_INVALID_ARG, missing
    assert call(starts=0x8002) == fa.FLEX_ERR_ALIGNMENT
    assert call(table=0x5002) == fa.FLEX_ERR_ALIGNMENT
    assert call(n=0) == fa.FLEX_ERR_SHAPE
    assert call(n=70000) == fa.FLEX_ERR_UNSUPPORTED
    assert call(width=-1) == fa.FLEX_ERR_SHAPE
    assert call(width=2**25) == fa.FLEX_ERR_UNSUPPORTED
    assert call(k=_tensor(BF, [2, 2, 5, 128])) == fa.FLEX_ERR_SHAPE
    assert call(k=_tensor(BF, [1, 2, 5, 64])) == fa.FLEX_ERR_SHAPE
    assert call(k=_tensor(BF, [1, 4, 5, 128])) == fa.FLEX_ERR_SHAPE
    assert call(v=_tensor(BF, [1, 2, 6, 128])) == fa.FLEX_ERR_SHAPE
    assert call(v=_tensor(F32, [1, 2, 5, 128])) == fa.FLEX_ERR_INVALID_ARG
    assert call(k=_tensor(E4, [1, 2, 5, 128])) == fa.FLEX_ERR_INVALID_ARG
    assert call(k=_tensor(BF, [1, 2, 5, 128], data=0x10008)) == fa.FLEX_ERR_ALIGNMENT
    assert call(k=_tensor(BF, [1, 2, 5, 128], stride=[1280, 640, 132, 1])) == fa.FLEX_ERR_ALIGNMENT


def test_python_refusals(lib):
    c = torch.zeros((4, 2, 16, 32), dtype=torch.uint8)
    ks, vs = torch.zeros((4, 2, 16, 2), dtype=torch.bfloat16), torch.zeros((4, 2, 16), dtype=torch.bfloat16)
    cache = fa.KVCache(c, c.clone(), ks, vs)
    assert cache.shape == (4, 2, 16, 64)
    for bad in ((c, c), (c, c, ks, None), (c, c, ks, ks), (c, c, vs, vs), (c, c, ks.float(), vs), (c, c[:3], ks, vs),
                (c, c, ks, torch.zeros((4, 2, 16, 1), dtype=torch.bfloat16)), (c.int(), c.int(), ks, vs)):
        with pytest.raises(ValueError):
            fa.KVCache(*bad)
    k = torch.zeros((1, 2, 5, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((3, 2), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    starts = torch.tensor([0, 1, 3, 5], dtype=torch.int32)
    good = dict(cache=cache, k=k, v=k, starts=starts, page_table=table, cache_lens=lens)
    for bad in (dict(starts=starts.long()), dict(starts=starts[:1]), dict(starts=starts[:3]), dict(starts=starts[None]),
                dict(starts=torch.zeros(8, dtype=torch.int32)[::2]), dict(page_table=table[:2]), dict(page_table=table[0]),
                dict(cache_lens=lens[:2]), dict(k=k.half(), v=k.half()), dict(k=k[0], v=k[0]),
                dict(inv_freq=torch.zeros(16))):
        with pytest.raises(ValueError):
            fa.flex_kv_cache_append_packed(**{**good, **bad})
    good = dict(cache=cache, page_table=table, starts=starts, total=5)
    for bad in (dict(total=None), dict(starts=starts[:3]), dict(page_table=table.long()), dict(dtype=torch.float16),
                dict(k_out=k[0]), dict(v_out=k.half()), dict(k_out=k, total=None)):
        with pytest.raises(ValueError):
            fa.flex_kv_cache_read(**{**good, **bad})


def test_structure_matches_the_header():
    """The scales' pointers keep their place in the structure."""
    assert fa.flex_kv_cache.k_scale.offset == 40 and ctypes.sizeof(fa.flex_kv_cache) == 56
