"""Softcap of the cache attention at caps of every size.

Bounds.  A score is a float32 sum of D exact products, off by (D + 8) 2^-24 of
the sum of their sizes; capping it moves it by at most 2^-19 of the capped
score more (by 2^-22 of the cap, from a quarter of the cap on), and passes the
other error on at most once.  lse is off by the largest of these, plus 2^-19 for
exponentials and sums; weights by twice it, and by 2^-11 (e4m3) or 2^-8 (bf16)
for their rounding; the result is rounded once, 2^-8.
"""
import pytest
import torch

from block_sparse_masked_blockmask_gb300 import flexattn as fa

pytestmark = pytest.mark.gpu
E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16


@pytest.mark.parametrize("dtype", [E4M3, BF16], ids=["e4m3", "bf16"])
@pytest.mark.parametrize("D,G", [(64, 3), (128, 12)])
@pytest.mark.parametrize("cap", [1e-44, 1e-38, 1e-3, 0.4, 2.0, 5.0, 30.0, 1e3, 1e4, 1e6, 1e7, 1e20, 3e38])
def test_cap(cap, D, G, dtype):
    n, page, H = 200, 32, 2
    gen = torch.Generator().manual_seed(D + G)
    cache = fa.flex_kv_cache_create(7, H, D, page, dtype)
    for x in (cache.k, cache.v):
        x.copy_(torch.randn(x.shape, generator=gen).mul(32 if dtype == E4M3 else 1))
    if dtype == E4M3:
        cache.k_scale.fill_(2.0**-5)
        cache.v_scale.fill_(2.0**-5)
    table = torch.arange(7, dtype=torch.int32, device="cuda")[None]
    q = torch.randn((1, H * G, 1, D), generator=gen)
    q[0, :G] *= 4.0          # scores to about 16 and, below, to 4
    q[0, -1] = 0.0           # scores of zero
    q = q.bfloat16().cuda()
    out, lse = fa.flex_kv_cache_attention(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                                          score_kind=fa.FLEX_SCORE_SOFTCAP, score_param=cap)
    cap = torch.tensor(cap, dtype=torch.float32).double().item()  # as it is passed
    s_k, s_v = (2.0**-5, 2.0**-5) if dtype == E4M3 else (1.0, 1.0)
    k, v = (x.double().transpose(1, 2).reshape(7 * page, H, D)[:n].transpose(0, 1).repeat_interleave(G, 0) * s
            for x, s in ((cache.k, s_k), (cache.v, s_v)))
    x = torch.einsum("hd,hnd->hn", q[0, :, 0].double(), k) * D**-0.5
    size = torch.einsum("hd,hnd->hn", q[0, :, 0].double().abs(), k.abs()) * D**-0.5
    s = cap * torch.tanh(x / cap)
    e_s = ((D + 8) * 2.0**-24 * size + 2.0**-19 * s.abs()).amax(-1)
    ref = torch.logsumexp(s, -1)
    assert ((lse[0, :, 0].double() - ref).abs() <= e_s + 2.0**-19 * (1 + ref.abs())).all()
    p = torch.softmax(s, -1)
    want, sizes = torch.einsum("hn,hnd->hd", p, v), torch.einsum("hn,hnd->hd", p, v.abs())
    bound = ((2.0**-11 if dtype == E4M3 else 2.0**-8) + 2 * e_s[:, None] + 2.0**-18) * sizes + 2.0**-8 * want.abs()
    if dtype == E4M3:  # weights below fp16's smallest step
        total = (s - s.amax(-1, keepdim=True)).exp().sum(-1, keepdim=True)
        bound += 2.0**-32 * n * 448 * s_v / total
    assert ((out[0, :, 0].double() - want).abs() <= bound).all()
