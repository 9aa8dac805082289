"""Window + sinks masks: what the host refuses (no GPU needed)."""
import ctypes

import pytest

from block_sparse_masked_blockmask_gb300 import _build, flexattn as fa
from test_abi import _call_create, _fwd, _mask_struct, _tensor


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load_library()


def test_refusals(lib):
    kind = fa.FLEX_MASK_WINDOW_SINKS
    assert _call_create(lib, kind, None) == fa.FLEX_ERR_INVALID_ARG
    assert _call_create(lib, kind, fa.flex_mask_params(-1, 0, None)) == fa.FLEX_ERR_INVALID_ARG
    assert _call_create(lib, kind, fa.flex_mask_params(4, -1, None)) == fa.FLEX_ERR_INVALID_ARG
    assert _call_create(lib, 6, fa.flex_mask_params(4, 1, None)) == fa.FLEX_ERR_INVALID_ARG
    q, k, v = (_tensor(fa.FLEX_DTYPE_BF16, [1, 2, 256, 64]) for _ in range(3))
    for params in ((-1, 0), (0, -1)):
        bm = _mask_struct(kind=kind)
        bm.params = fa.flex_mask_params(*params, None)
        assert _fwd(lib, q, k, v, bm) == fa.FLEX_ERR_INVALID_ARG


def test_sinks_need_their_kind():
    with pytest.raises(ValueError):
        fa._mask_params(fa.FLEX_MASK_SLIDING_WINDOW, 4, 0, 2)
    p = fa._mask_params(fa.FLEX_MASK_WINDOW_SINKS, 4, 9, 2)
    assert (p.window, p.prefix) == (4, 2)
    assert ctypes.sizeof(fa.flex_mask_params) == 16
