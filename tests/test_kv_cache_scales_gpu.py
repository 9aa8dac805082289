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


def attended(q, cache, table, n, G, first=0):
    """float64 result of the causal attention of Q newest tokens of one sequence, and its bound.

    Scores are float32 sums of D products, off by (D + 8) 2^-24 of the sum of
    their sizes.  A weight is rounded to fp16, 2^-11 of itself, or half of
    fp16's smallest step, 2^-25 in units where the row's largest weight is 2^7
    at least and V is taken relative to a scale at most 2^6 times its page's:
    2^-26 of the row's largest, times 448 scales.  The result is rounded once.
    """
    Q, D, page = q.shape[2], q.shape[3], cache.k.shape[2]
    at = torch.arange(n, device="cuda")
    ids, slot = table[0].long()[at // page], at % page
    vs = cache.v_scale[ids].double().T                                  # [H, n]
    k = cache.k[ids, :, slot].double().transpose(0, 1) * cache.k_scale[ids].double().T[..., None]
    v = cache.v[ids, :, slot].double().transpose(0, 1) * vs[..., None]
    k, v, vs = (x.repeat_interleave(G, 0) for x in (k, v, vs))
    out, bound = (torch.zeros(q.shape[1:], dtype=torch.float64, device="cuda") for _ in range(2))
    for t in range(Q):
        m = n - Q + t + 1
        s = torch.einsum("hd,hnd->hn", q[0, :, t].double(), k[:, :m]) * D**-0.5
        size = torch.einsum("hd,hnd->hn", q[0, :, t].abs().double(), k[:, :m].abs()) * D**-0.5
        p = torch.softmax(s, -1)
        e_s = (D + 8) * 2.0**-24 * size.amax(-1, keepdim=True)
        total = (s - s.amax(-1, keepdim=True)).exp().sum(-1, keepdim=True)
        out[:, t] = torch.einsum("hn,hnd->hd", p, v[:, :m])
        bound[:, t] = (2.0**-11 + 2 * e_s + 2.0**-18) * torch.einsum("hn,hnd->hd", p, v[:, :m].abs()) + \
            2.0**-26 * 448 * vs[:, :m].sum(-1, keepdim=True) / total + 2.0**-8 * out[:, t].abs()
    return out, bound


def scaled_cache(gen, n, page, D, H, big, scale):
    """One sequence of n tokens with V scales of 2^-8, but `scale` on page `big` of the table."""
    pages = -(-n // page)
    cache = fa.flex_kv_cache_create(pages, H, D, page, E4M3)
    cache.k.copy_(torch.randn(cache.k.shape, generator=gen).mul(64).clamp(-448, 448))
    cache.v.copy_(torch.randn(cache.v.shape, generator=gen).mul(100).clamp(-448, 448))
    table = torch.randperm(pages, generator=gen).int().cuda()[None]
    cache.k_scale.fill_(2.0**-6)
    cache.v_scale.fill_(2.0**-8)
    cache.v_scale[table[0, big].long()] = scale
    return cache, table


EXPONENTS = (-90, -13, -3, 2, 12, 20, 23, 32, 50, 80)


@pytest.mark.parametrize("G,page,D,n", [(1, 16, 64, 97), (4, 64, 128, 257), (3, 32, 128, 193), (8, 64, 64, 129),
                                        (2, 16, 128, 3009), (4, 128, 64, 5121)])
def test_scale_of_a_page_that_a_row_does_not_keep(G, page, D, n):
    """Two tokens, the second alone on a page of any V scale: the first gets what it gets without that page."""
    gen = torch.Generator().manual_seed(n + D)
    for e in EXPONENTS:
        cache, table = scaled_cache(gen, n, page, D, 2, -1, 2.0**e)
        q = torch.randn((1, 2 * G, 2, D), generator=gen).bfloat16().cuda()
        out, _ = fa.flex_kv_cache_attention(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
        want, bound = attended(q, cache, table, n, G)
        assert ((out[0].double() - want).abs() <= bound).all(), e


@pytest.mark.parametrize("where", [0, 1, -1])
@pytest.mark.parametrize("G,page,D,n", [(1, 16, 64, 96), (4, 64, 128, 256), (16, 32, 128, 192), (2, 16, 128, 3008),
                                        (8, 128, 64, 5120)])
def test_scale_of_a_page_without_weight(G, page, D, n, where):
    """A page of any V scale that no query looks at (scores 200 below the others'): the others' share is what counts."""
    gen = torch.Generator().manual_seed(n + D + where)
    for e in EXPONENTS:
        cache, table = scaled_cache(gen, n, page, D, 2, where, 2.0**e)
        pid = int(table[0, where])
        cache.k[:, :, :, 0] = torch.tensor(64.0, device="cuda").to(E4M3)     # 1, and -8 on that page
        cache.k_scale[pid] = 2.0**-3
        cache.k[pid, :, :, 0] = torch.tensor(-64.0, device="cuda").to(E4M3)
        cache.k[pid, :, :, 1:] = torch.zeros((), device="cuda").to(E4M3)
        q = torch.randn((1, 2 * G, 1, D), generator=gen)
        q[..., 0] = 200.0 * D**0.5 / 9
        q = q.bfloat16().cuda()
        out, _ = fa.flex_kv_cache_attention(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
        want, bound = attended(q, cache, table, n, G)
        # weights of e^-200 leave nothing of any scale here, beside the bound's terms for them
        live = torch.arange(n, device="cuda") // page != where % (-(-n // page))
        lone = cache.v_scale.clone()
        cache.v_scale[pid] = 0.0
        want, bound = attended(q, cache, table, n, G)
        cache.v_scale.copy_(lone)
        assert live.any() and 2.0**e * 448 * math.exp(-199) < 2.0**-149
        assert ((out[0].double() - want).abs() <= bound).all(), e


def test_scale_beside_a_value_that_is_not_finite():
    """Three tokens, the last two on a page of a large V scale, the last one with a NaN: rows that do not keep it."""
    G, page, D, n = 2, 16, 64, 98
    gen = torch.Generator().manual_seed(4)
    for e in EXPONENTS:
        cache, table = scaled_cache(gen, n, page, D, 2, -1, 2.0**e)
        q = torch.randn((1, 2 * G, 3, D), generator=gen).bfloat16().cuda()
        want, bound = attended(q, cache, table, n, G)
        cache.v[int(table[0, -1]), :, 1, 5] = torch.tensor(math.nan, device="cuda").to(E4M3)
        out, _ = fa.flex_kv_cache_attention(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
        assert out[0, :, 2, 5].isnan().all()
        diff = (out[0].double() - want).abs() <= bound
        diff[:, 2, 5] = True
        assert diff.all(), e


@pytest.mark.parametrize("n,B,H,G,Q", [(700, 2, 2, 4, 1), (5000, 40, 8, 4, 1), (130, 3, 2, 5, 7), (3000, 1, 1, 16, 2)])
def test_result_in_place_of_the_queries(n, B, H, G, Q):
    gen = torch.Generator().manual_seed(n)
    D, page = 128, 64
    width = -(-n // page)
    cache = fa.flex_kv_cache_create(width, H, D, page, E4M3)
    cache.k.copy_(torch.randn(cache.k.shape, generator=gen))
    cache.v.copy_(torch.randn(cache.v.shape, generator=gen))
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    table = torch.arange(width, dtype=torch.int32, device="cuda").expand(B, width).contiguous()
    lens = torch.randint(1, n + 1, (B,), generator=gen).int().cuda()
    q = torch.randn((B, H * G, Q, D), generator=gen).bfloat16().cuda()
    out, lse = fa.flex_kv_cache_attention(q, cache, table, lens)
    again, l2 = fa.flex_kv_cache_attention(q, cache, table, lens, out=q)
    assert again is q and torch.equal(out, q) and torch.equal(lse, l2)
