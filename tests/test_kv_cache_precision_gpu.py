"""The cache attention at the precision that its weights have.

Bounds.  Scores are float32 sums of D products, off by (D + 8) 2^-24 of the sum
of their sizes; lse by the largest of these, plus 2^-19 for exponentials and
sums.  A weight is rounded to fp16 (e4m3 cache: 2^-11) or bf16 (2^-8).  In fp16 it
is also off by half of the smallest step, 2^-25, in units in which the row's
largest weight is 2^7 at least and a page's weights are relative to a V scale that
is at most 2^6 times its own, and at most the largest: 2^-32 of the row's largest,
times min(the largest V scale, 2^6 of its own), times its value / scale.  The
result is rounded once, 2^-8.
"""
import math

import pytest
import torch

from block_sparse_masked_blockmask_gb300 import flexattn as fa
from test_kv_cache_gpu import BF16, E4M3, filled, values

pytestmark = pytest.mark.gpu


def check(q, cache, table, lens, kind, window, sinks, score, cap):
    n_ = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = fa.flex_kv_cache_attention(q, cache, table, n_, kind, window, sinks, score, cap)
    B, Hq, Q, D = q.shape
    page, G = cache.k.shape[2], Hq // cache.k.shape[1]
    e4m3 = cache.k.dtype == E4M3
    kd, vd = values(cache, "k"), values(cache, "v")
    slope = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float64) / Hq)
    for b, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        ids, slot = table[b].long()[at // page], at % page
        k, v = (x[ids, :, slot].transpose(0, 1).repeat_interleave(G, 0) for x in (kd, vd))
        vs = cache.v_scale[ids].double().T.repeat_interleave(G, 0) if e4m3 else None
        for t in range(Q):
            pos = n - Q + t
            keep = at <= pos if kind != fa.FLEX_MASK_ALL else torch.full_like(at, pos >= 0, dtype=torch.bool)
            if kind in (fa.FLEX_MASK_SLIDING_WINDOW, fa.FLEX_MASK_WINDOW_SINKS):
                keep &= (pos - at < window) | (at < sinks)
            if not keep.any():
                assert (out[b, :, t] == 0).all() and torch.isneginf(lse[b, :, t]).all()
                continue
            s = torch.einsum("hd,hnd->hn", q[b, :, t].double(), k[:, keep]) * D**-0.5
            size = torch.einsum("hd,hnd->hn", q[b, :, t].double().abs(), k[:, keep].abs()) * D**-0.5
            if score == fa.FLEX_SCORE_SOFTCAP:
                s = cap * torch.tanh(s / cap)
                size = size + 2.0**5 / (D + 8) * s.abs()  # 2^-19 of it
            elif score == fa.FLEX_SCORE_ALIBI:
                far = slope[:, None] * (pos - at[keep]).double()
                s, size = s - far, size + far.abs()
            # an error of a score counts with its weight
            p = torch.softmax(s, -1)
            e = (D + 8) * 2.0**-24 * size
            e_l = (p * e).sum(-1) * 1.01 + 2.0**-19 * (1 + torch.logsumexp(s, -1).abs())
            assert ((lse[b, :, t].double() - torch.logsumexp(s, -1)).abs() <= e_l).all()
            want = torch.einsum("hn,hnd->hd", p, v[:, keep])
            off = p * ((2.0**-11 if e4m3 else 2.0**-8) + e * 1.01 + e_l[:, None] + 2.0**-18)
            if e4m3:
                total = (s - s.amax(-1, keepdim=True)).exp().sum(-1, keepdim=True)
                mine = vs[:, keep]
                ref = torch.minimum(mine.amax(-1, keepdim=True), 64 * mine)
                off = off + 2.0**-32 * ref / mine / total
            bound = torch.einsum("hn,hnd->hd", off, v[:, keep].abs()) + 2.0**-8 * want.abs()
            diff = (out[b, :, t].double() - want).abs()
            assert (diff <= bound).all(), (b, t, float((diff / bound).max()))


@pytest.mark.parametrize("dtype", [E4M3, BF16], ids=["e4m3", "bf16"])
@pytest.mark.parametrize("H,G,Q,D,page,lens", [(2, 4, 1, 128, 64, [1, 0, 700, 130]), (1, 3, 5, 64, 16, [3, 300, 64]),
                                               (2, 8, 2, 128, 16, [257, 40]), (1, 16, 1, 64, 128, [500, 129]),
                                               (4, 4, 1, 128, 64, [9000, 4001]), (2, 8, 4, 64, 256, [5000]),
                                               (1, 5, 7, 128, 32, [2, 1000])])
def test_bounds(H, G, Q, D, page, lens, dtype):
    gen = torch.Generator().manual_seed(D + page + 7 * H * G * Q)
    cache, table = filled(gen, lens, H, page, D, dtype)
    q = torch.randn((len(lens), H * G, Q, D), generator=gen).bfloat16().cuda()
    for kind, window, sinks, score in ((fa.FLEX_MASK_CAUSAL, 0, 0, fa.FLEX_SCORE_IDENTITY),
                                       (fa.FLEX_MASK_WINDOW_SINKS, 100, 4, fa.FLEX_SCORE_IDENTITY),
                                       (fa.FLEX_MASK_SLIDING_WINDOW, 33, 0, fa.FLEX_SCORE_SOFTCAP),
                                       (fa.FLEX_MASK_CAUSAL, 0, 0, fa.FLEX_SCORE_ALIBI),
                                       (fa.FLEX_MASK_ALL, 0, 0, fa.FLEX_SCORE_SOFTCAP)):
        check(q, cache, table, lens, kind, window, sinks, score, 5.0)


@pytest.mark.parametrize("at", [5, 61])
@pytest.mark.parametrize("G,D", [(1, 64), (4, 128), (16, 128)])
@pytest.mark.parametrize("less", [10.0, 14.0, 18.0])
def test_many_small_weights_beside_large_ones(less, G, D, at):
    """In every page one token with nearly all of the weight and a value of zero; the others, at e^-10 to e^-18 of it,
    are the only ones with values: their sum is what comes out."""
    n, page = 20000, 64
    pages = -(-n // page)
    cache = fa.flex_kv_cache_create(pages, 1, D, page, E4M3)
    cache.k.copy_(torch.zeros(cache.k.shape))
    cache.v.copy_(torch.full(cache.v.shape, 448.0))
    cache.k_scale.fill_(2.0**-8)
    cache.v_scale.fill_(2.0**-8)
    cache.k[:, 0, at, 0] = torch.tensor(256.0, device="cuda").to(E4M3)  # 1
    cache.v[:, 0, at] = torch.zeros((), device="cuda").to(E4M3)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    q = torch.zeros((1, G, 1, D))
    q[..., 0] = less * math.sqrt(D)
    check(q.bfloat16().cuda(), cache, table, [n], fa.FLEX_MASK_CAUSAL, 0, 0, fa.FLEX_SCORE_IDENTITY, 0.0)
