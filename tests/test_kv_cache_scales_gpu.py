"""Scales of the paged e4m3 cache that the append did not write itself.

Bounds.  A code is within half a step of value / scale: 2^-4 of itself, or
2^-10 (half of e4m3's smallest step) below 2^-6.  The quotient is a float32
product with a reciprocal, two roundings of 2^-24 before that of the code:
2^-22 of the value covers them.
"""
import math

import pytest
import torch

from block_sparse_masked_blockmask_gb300 import flexattn as fa

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32], ids=["from_bf16", "from_fp32"])
@pytest.mark.parametrize("page,D,S", [(64, 128, 1), (64, 128, 40), (256, 64, 150), (16, 64, 3)])
@pytest.mark.parametrize("held", [1.5, 1.25, 0.01, 3e-3, 1e-6, 2.0**-5, 1e30])
def test_append_to_a_page_of_another_scale(held, page, D, S, src):
    """A page half full of codes under any scale: it is kept where the new tokens fit, else becomes their power of two,
    and old and new values are what they were to half a step."""
    H, old_n = 3, page // 2
    gen = torch.Generator().manual_seed(page + S)
    width = -(-(old_n + S) // page)
    cache = fa.flex_kv_cache_create(width, H, D, page, E4M3)
    codes = torch.randn((2, H, old_n, D), generator=gen).mul(100).clamp(-448, 448).to(E4M3).cuda()
    for x, c in ((cache.k, codes[0]), (cache.v, codes[1])):
        x.copy_(torch.zeros(x.shape))
        x[0, :, :old_n] = c
    for s in (cache.k_scale, cache.v_scale):
        s.fill_(math.nan)
        s[0] = held * torch.tensor([1.0, 1.1, 0.7], device="cuda")
    before = [s[0].double() for s in (cache.k_scale, cache.v_scale)]
    k, v = (torch.randn((1, H, S, D), generator=gen).to(src).cuda() for _ in range(2))
    fa.flex_kv_cache_append(cache, k, v, torch.arange(width, dtype=torch.int32, device="cuda")[None],
                            torch.tensor([old_n], dtype=torch.int32, device="cuda"))
    here = min(S, page - old_n)  # new tokens on the page
    for x, c, s, sc, got in zip((k, v), codes, before, (cache.k_scale, cache.v_scale), (cache.k, cache.v)):
        new = x[0, :, :here].double()
        amax = new.abs().amax((1, 2))
        now = sc[0].double()
        # the smallest power of two s with amax <= 448 s: 224 s < amax
        raised = amax > 448 * s
        assert torch.equal(now[~raised], torch.maximum(s, now)[~raised])
        lone = now != s
        mantissa, _ = torch.frexp(now)
        assert ((mantissa == 0.5) & (amax <= 448 * now) & (224 * now < amax) & (now > s))[lone].all()
        assert lone[raised].all()
        step = lambda y: torch.maximum(2.0**-4 * y.abs(), (now * 2.0**-10)[:, None, None])  # noqa: E731
        y = got[0, :, old_n:old_n + here].double() * now[:, None, None]
        assert ((y - new).abs() <= step(new) + 2.0**-22 * new.abs()).all()
        y, want = got[0, :, :old_n].double() * now[:, None, None], c.double() * s[:, None, None]
        assert ((y - want).abs() <= torch.where(lone[:, None, None], step(want) + 2.0**-22 * want.abs(), 0.0)).all()


def test_appended_page_of_another_scale_is_attended():
    """What the attention reads back of such a page is what was appended: one token looks at itself alone."""
    H, D, page = 2, 64, 16
    cache = fa.flex_kv_cache_create(1, H, D, page, E4M3)
    for x in (cache.k, cache.v):
        x.copy_(torch.zeros(x.shape))
    cache.k_scale.fill_(1.5)
    cache.v_scale.fill_(1.25)
    gen = torch.Generator().manual_seed(2)
    x = torch.randn((1, H, 1, D), generator=gen).mul(100).bfloat16().cuda()
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    n = torch.tensor([7], dtype=torch.int32, device="cuda")
    fa.flex_kv_cache_append(cache, x, x, table, n)
    out, _ = fa.flex_kv_cache_attention(x, cache, table, n + 1, fa.FLEX_MASK_SLIDING_WINDOW, 1)
    # a half step of the code, the weight of fp16 and the last rounding
    bound = 2.0**-4 * x.abs().double() + 1.25 * 2.0**-10 + (2.0**-11 + 2.0**-8) * x.abs().double() * 1.0625
    assert ((out.double() - x.double()).abs() <= bound).all()
