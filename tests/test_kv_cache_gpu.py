"""The paged key/value cache: appends against a float64 restatement of the
page's rule, attention against the formula in float64 over the cache's values,
and both together as a decoding loop.

Bounds.  A code is within half a step of value / scale: 2^-4 of itself, or
2^-10 (half of e4m3's smallest step) below 2^-6; a rotated key adds 2^-20 of
its pair (the fast sine and cosine).  A re-rounded code is off by another half
step of the new scale.  Scores of the attention are float32 sums of D exact
products: off by at most (D + 8) 2^-24 scale sum |q k|, and so is lse (plus
2^-19 for exponentials and sums).  Weights are rounded to fp16 (e4m3 cache:
2^-11) or bf16 (2^-8), or fall below fp16's smallest step, 2^-25 of the
largest weight (at least 2^-8 of 1 in the kernel's units) times the largest V
scale; out is rounded once, 2^-8.
"""
import math
import os
import subprocess
import sys

import pytest
import torch

from block_sparse_masked_blockmask_gb300 import flexattn as fa

pytestmark = pytest.mark.gpu
E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16


def power_scale(amax):
    """Smallest power of two s >= 2^-126 with amax <= 448 s, in float64."""
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, 2.0**-130) / 448.0)).clamp(min=-126.0)
    s = ((e.long() + 1023) << 52).view(torch.float64)  # 2^e exactly, which pow need not be
    s = torch.where(amax > 448.0 * s, 2 * s, s)
    return torch.where((amax <= 224.0 * s) & (s > 2.0**-126), s / 2, s)


def table_of(gen, counts, width, extra=3):
    """Pages in random order for every sequence, -1 behind; the number of pages."""
    total = sum(counts)
    order = torch.randperm(total + extra, generator=gen)[:total].to(torch.int32)
    t = torch.full((len(counts), width), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        t[b, :c] = order[at:at + c]
        at += c
    return t.cuda(), total + extra


def new_cache(pages, H, page, D, dtype, fill=float("nan")):
    c = fa.flex_kv_cache_create(pages, H, D, page, dtype)
    for x in (c.k, c.v):
        x.copy_(torch.full(x.shape, fill, device="cuda"))  # slots never written hold NaN
    if dtype == E4M3:
        c.k_scale.fill_(float("nan"))
        c.v_scale.fill_(float("nan"))
    return c


def rotated(x, pos, inv, layout):
    r = 2 * inv.numel()
    y, size = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    a, b = (slice(0, r // 2), slice(r // 2, r)) if layout == fa.FLEX_ROPE_HALF else (slice(0, r, 2), slice(1, r, 2))
    angle = pos.double()[:, None] * inv
    z = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.ones_like(angle), angle)
    size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
    y[..., a], y[..., b] = z.real, z.imag
    return y, size


def values(cache, which):
    x = getattr(cache, which).double()
    s = getattr(cache, which + "_scale")
    return x if s is None else x * s.double()[:, :, None, None]


@pytest.mark.parametrize("dtype", [E4M3, BF16], ids=["e4m3", "bf16"])
@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32], ids=["from_bf16", "from_fp32"])
@pytest.mark.parametrize("page,D,rotary,layout", [(16, 64, 16, fa.FLEX_ROPE_HALF), (64, 128, 128, fa.FLEX_ROPE_INTERLEAVED),
                                                  (256, 128, 64, fa.FLEX_ROPE_HALF), (32, 64, 0, fa.FLEX_ROPE_HALF)])
def test_append(page, D, rotary, layout, src, dtype):
    """Several appends of odd lengths, ragged: every page's scale, codes, and what must stay as it was."""
    H, B = 3, 4
    gen = torch.Generator().manual_seed(page + D)
    calls = [(5, [5, 0, 3, 5]), (1, None), (37, [37, 20, 0, 9]), (1, [1, 1, 0, 1]), (300, [300, 1, 290, 7]), (1, None)]
    width = -(-400 // page)
    table, pages = table_of(gen, [width] * B, width)
    cache = new_cache(pages, H, page, D, dtype)
    inv = fa.flex_rope_frequencies(rotary) if rotary else None
    lens = torch.zeros(B, dtype=torch.int32)
    want = {w: torch.full((pages, H, page, D), math.nan, dtype=torch.float64, device="cuda") for w in "kv"}
    slack = {w: torch.zeros((pages, H, page, D), dtype=torch.float64, device="cuda") for w in "kv"}
    scale = {w: torch.zeros((pages, H), dtype=torch.float64, device="cuda") for w in "kv"}
    for n, (S, new) in enumerate(calls):
        # sizes that grow and shrink from call to call, so that scales rise within a page
        k, v = (torch.randn((B, S, H, D), generator=gen).mul(4.0 ** ((n * 3) % 5 - 2)).to(src).cuda().transpose(1, 2)
                for _ in range(2))
        fa.flex_kv_cache_append(cache, k, v, table, lens.cuda(), None if new is None else torch.tensor(new).int().cuda(),
                                inv_freq=inv, layout=layout)
        for b in range(B):
            count = S if new is None else new[b]
            pos = lens[b] + torch.arange(count)
            for w, x in (("k", k), ("v", v)):
                y, size = x[b, :, :count].double(), 0.0
                if w == "k" and rotary:
                    y, size = rotated(x[b, :, :count], pos.cuda(), inv, layout)
                    size = size * 2.0**-20
                ids, at = table[b].long()[(pos // page).cuda()], (pos % page).cuda()
                for i in ids.unique().tolist():
                    mine = ids == i
                    want[w][i, :, at[mine]] = y[:, mine]
                    if dtype == E4M3:
                        grown = power_scale(y[:, mine].abs().amax((1, 2)))
                        if int(at[mine][0]) > 0:
                            grown = torch.maximum(grown, scale[w][i])
                        held = torch.arange(page, device="cuda") < at[mine][0]
                        again = (grown > scale[w][i])[:, None] & held
                        # a code that is rounded once more: half a step of the new scale
                        slack[w][i] += torch.where(again[..., None], grown[:, None, None] * 2.0**-10, 0.0)
                        scale[w][i] = grown
                        slack[w][i, :, at[mine]] = torch.zeros((), dtype=torch.float64, device="cuda")
                    if isinstance(size, torch.Tensor):
                        slack[w][i, :, at[mine]] += size[:, mine]
        lens += S if new is None else torch.tensor(new).int()
        for w in "kv":
            got, ref = values(cache, w), want[w]
            written = ~ref.isnan()
            assert got.isnan()[~written].all(), (n, w, "a slot without a token was written")
            diff = (got - ref).abs()
            if dtype == E4M3:
                used = written.any(3).any(2)
                sc = getattr(cache, w + "_scale")
                assert torch.equal(sc.double()[used], scale[w][used]), (n, w, "scale")
                # half a step at the value, or of the smallest steps
                bound = torch.maximum(2.0**-4 * ref.abs(), (scale[w] * 2.0**-10)[:, :, None, None]) + slack[w] * 1.0625
            else:
                bound = 2.0**-8 * ref.abs() + slack[w]
            bad = written & (diff > bound)
            assert not bad.any(), (n, w, float(diff[bad].max()))


def test_append_leaves_alone_and_drops():
    """Bad pages, tokens past the table, negative lengths, sequences without new tokens, infinities and zeros."""
    H, D, page = 2, 64, 16
    cache = new_cache(6, H, page, D, E4M3)
    before = cache.k.view(torch.uint8).clone()
    k = torch.ones((6, H, 20, D), device="cuda").bfloat16()
    table = torch.tensor([[-1, 0], [6, 1], [2, -7], [3, 100], [4, 5], [4, 5]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([0, 0, 0, 30, -1, 40], dtype=torch.int32, device="cuda")
    new = torch.tensor([20, 20, 18, 20, 20, 20], dtype=torch.int32, device="cuda")
    fa.flex_kv_cache_append(cache, k, k, table, lens, new)
    torch.cuda.synchronize()
    got = cache.k.view(torch.uint8)
    changed = (got != before).any(3).any(1)
    want = torch.zeros((6, page), dtype=torch.bool)
    want[0, :4] = want[1, :4] = True   # the second page of sequences whose first is bad
    want[2, :] = True
    assert torch.equal(changed.cpu(), want)
    # non-finite values: code NaN, no part in the scale; a page of zeros
    cache = new_cache(2, H, page, D, E4M3)
    x = torch.zeros((1, H, 17, D), device="cuda")
    x[0, 0, 16, 3], x[0, 0, 16, 4], x[0, 0, 16, 5] = math.inf, math.nan, 3.5
    fa.flex_kv_cache_append(cache, x, x, torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"),
                            torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert (cache.v_scale[1] == 2.0**-126).all() and (cache.v[1].float() == 0).all()
    assert cache.v_scale[0, 0] == 2.0**-7 and cache.v[0, 0, 0, 5].float() == 448
    assert cache.v[0, 0, 0, 3:5].float().isnan().all()
    assert cache.v[0, 0, 0].float().isnan().sum() == 2


def filled(gen, lens, H, page, D, dtype, extra_width=2):
    """A cache with random contents for these lengths; free pages and free slots hold NaN (and NaN scales)."""
    counts = [-(-n // page) for n in lens]
    width = max(1, max(counts)) + extra_width
    table, pages = table_of(gen, counts, width)
    cache = new_cache(pages, H, page, D, dtype)
    for b, n in enumerate(lens):
        for i in range(counts[b]):
            used = min(page, n - i * page)
            pid = int(table[b, i])
            for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
                y = torch.randn((H, used, D), generator=gen).cuda()
                if dtype == E4M3:
                    sc = 2.0 ** torch.randint(-12, 3, (H,), generator=gen).float().cuda()
                    s[pid] = sc
                    y = y * torch.where(sc < 0.01, 448.0 / 4, 1.0)[:, None, None]  # some pages use the whole range
                x[pid, :, :used] = y.clamp(-448.0, 448.0).to(dtype)
    return cache, table


def reference(q, cache, table, lens, page, kind, window, sinks, score, cap, scale):
    """float64 out, lse, and bounds of both."""
    B, Hq, Q, D = q.shape
    H = cache.k.shape[1]
    G = Hq // H
    out = torch.zeros((B, Hq, Q, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Q), -math.inf, dtype=torch.float64, device="cuda")
    bo, bl = torch.zeros_like(out), torch.zeros_like(lse)
    kd, vd = values(cache, "k"), values(cache, "v")
    slope = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float64) / Hq)
    for b, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        ids = table[b].long()[at // page]
        good = (ids >= 0) & (ids < cache.k.shape[0])
        ids = ids.clamp(0, cache.k.shape[0] - 1)
        for t in range(Q):
            pos = n - Q + t
            if pos < 0:
                continue
            keep = good.clone()
            if kind != fa.FLEX_MASK_ALL:
                keep &= at <= pos
            if kind in (fa.FLEX_MASK_SLIDING_WINDOW, fa.FLEX_MASK_WINDOW_SINKS):
                keep &= (pos - at < window) | (at < sinks)
            idx = keep.nonzero()[:, 0]
            if not len(idx):
                continue
            k, v = (x[ids[idx], :, idx % page].transpose(0, 1) for x in (kd, vd))   # [H, n, D]
            qt = q[b, :, t].double().reshape(H, G, D)
            s = torch.einsum("hgd,hnd->hgn", qt, k) * scale
            size = torch.einsum("hgd,hnd->hgn", qt.abs(), k.abs()) * abs(scale)
            if score == fa.FLEX_SCORE_SOFTCAP:
                s = cap * torch.tanh(s / cap)
            elif score == fa.FLEX_SCORE_ALIBI:
                far = slope.reshape(H, G, 1) * (pos - idx).double()
                s, size = s - far, size + far.abs()
            p = torch.softmax(s, -1)
            lse[b, :, t] = torch.logsumexp(s, -1).reshape(-1)
            out[b, :, t] = torch.einsum("hgn,hnd->hgd", p, v).reshape(Hq, D)
            e_s = ((D + 8) * 2.0**-24 * size.amax(-1)).reshape(-1)
            bl[b, :, t] = e_s + 2.0**-19 * (1 + lse[b, :, t].abs())
            absolute = torch.einsum("hgn,hnd->hgd", p, v.abs()).reshape(Hq, D)
            r = 2.0**-11 if cache.k.dtype == E4M3 else 2.0**-8
            bo[b, :, t] = (r + 2 * e_s[:, None] + 2.0**-18) * absolute + 2.0**-8 * out[b, :, t].abs()
            if cache.k.dtype == E4M3:
                # each weight below fp16's smallest step: 2^-25 of 448 V scales, in units in which the row's sum is
                # at least 2^-8 (the running maximum may trail by 2^8)
                total = torch.exp(torch.logsumexp(s, -1) - s.amax(-1)).reshape(-1)
                top = 448 * cache.v_scale[ids[idx]].double().amax(0).repeat_interleave(G)
                bo[b, :, t] += (2.0**-25 * len(idx) * top / total)[:, None]
    return out, lse, bo, bl


def compare(q, cache, table, lens, page, kind=fa.FLEX_MASK_CAUSAL, window=0, sinks=0, score=fa.FLEX_SCORE_IDENTITY,
            cap=5.0, scale=None):
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
    out, lse = fa.flex_kv_cache_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), kind,
                                          window, sinks, score, cap, scale)
    ro, rl, bo, bl = reference(q, cache, table, lens, page, kind, window, sinks, score, cap, scale)
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), empty) and (out[empty] == 0).all()
    assert (torch.where(empty, 0.0, lse.double() - rl).abs() <= bl).all(), \
        float(torch.where(empty, 0.0, lse.double() - rl).abs().max())
    diff = (out.double() - ro).abs()
    assert (diff <= bo).all(), float((diff - bo).max())
    return out, lse


MASKS = [(fa.FLEX_MASK_CAUSAL, 0, 0), (fa.FLEX_MASK_SLIDING_WINDOW, 5, 0), (fa.FLEX_MASK_SLIDING_WINDOW, 0, 0),
         (fa.FLEX_MASK_WINDOW_SINKS, 33, 4), (fa.FLEX_MASK_WINDOW_SINKS, 1, 70), (fa.FLEX_MASK_WINDOW_SINKS, 0, 3),
         (fa.FLEX_MASK_WINDOW_SINKS, 2**31 - 1, 2**31 - 1), (fa.FLEX_MASK_ALL, 0, 0)]


@pytest.mark.parametrize("dtype", [E4M3, BF16], ids=["e4m3", "bf16"])
@pytest.mark.parametrize("D,page", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 256)])
@pytest.mark.parametrize("H,G,Q", [(1, 1, 1), (2, 4, 1), (1, 8, 2), (2, 3, 5), (1, 1, 9), (1, 17, 1), (1, 5, 7)])
def test_attention(H, G, Q, D, page, dtype):
    lens = [1, 0, 17, 130, 300, 64, 3]
    gen = torch.Generator().manual_seed(D + page + 7 * H * G * Q)
    cache, table = filled(gen, lens, H, page, D, dtype)
    q = torch.randn((len(lens), Q, H * G, D), generator=gen).bfloat16().cuda().transpose(1, 2)
    scores = (fa.FLEX_SCORE_IDENTITY, fa.FLEX_SCORE_SOFTCAP, fa.FLEX_SCORE_ALIBI)
    for i, (kind, window, sinks) in enumerate(MASKS):
        compare(q, cache, table, lens, page, kind, window, sinks, scores[i % 3])


@pytest.mark.parametrize("dtype", [E4M3, BF16], ids=["e4m3", "bf16"])
@pytest.mark.parametrize("lens,G,Q", [([20000], 8, 1), ([3000, 1, 2999], 2, 1), ([5000], 4, 33)])
def test_attention_long(lens, G, Q, dtype):
    gen = torch.Generator().manual_seed(lens[0])
    cache, table = filled(gen, lens, 2, 64, 128, dtype)
    q = torch.randn((len(lens), 2 * G, Q, 128), generator=gen).bfloat16().cuda()
    compare(q, cache, table, lens, 64)
    compare(q, cache, table, lens, 64, fa.FLEX_MASK_WINDOW_SINKS, 1000, 5, fa.FLEX_SCORE_ALIBI)


@pytest.mark.parametrize("D,G,Q,dtype", [(128, 4, 1, E4M3), (128, 1, 1, BF16), (64, 8, 1, E4M3), (64, 2, 2, BF16),
                                         (128, 4, 3, E4M3), (64, 16, 1, BF16)], ids=str)
def test_attention_many_steps(D, G, Q, dtype):
    """A ragged batch large enough that every warp of the launch walks over many steps, sequences and heads."""
    gen = torch.Generator().manual_seed(D + G)
    B, H, page = 40, 8, 64
    lens = torch.randint(1, 9000, (B,), generator=gen).tolist()
    lens[3], lens[4], lens[20] = 0, 1, 9000
    cache, table = filled(gen, lens, H, page, D, dtype)
    q = torch.randn((B, H * G, Q, D), generator=gen).bfloat16().cuda()
    compare(q, cache, table, lens, page)


@pytest.mark.parametrize("B,dtype", [(129, E4M3), (300, BF16), (1000, E4M3)], ids=str)
def test_attention_many_sequences(B, dtype):
    """More sequences than a CTA has threads: the list's prefix sums and the search in them."""
    gen = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 90, (B,), generator=gen).tolist()
    cache, table = filled(gen, lens, 2, 32, 64, dtype)
    q = torch.randn((B, 4, 2, 64), generator=gen).bfloat16().cuda()
    compare(q, cache, table, lens, 32)
    compare(q, cache, table, lens, 32, fa.FLEX_MASK_WINDOW_SINKS, 10, 3)


@pytest.mark.parametrize("dtype", [E4M3, BF16], ids=["e4m3", "bf16"])
def test_attention_shared_and_bad_pages(dtype):
    """Two sequences on the same pages; entries that name no page are masked; entries behind a window are not read."""
    gen = torch.Generator().manual_seed(9)
    lens = [200, 150, 180]
    cache, table = filled(gen, lens, 2, 32, 64, dtype)
    table[1, :5] = table[0, :5]
    table[2, 1], table[2, 3] = -1, cache.k.shape[0]
    q = torch.randn((3, 4, 2, 64), generator=gen).bfloat16().cuda()
    compare(q, cache, table, lens, 32)
    a = compare(q, cache, table, lens, 32, fa.FLEX_MASK_WINDOW_SINKS, 40, 2)
    for b, n in enumerate(lens):
        table[b, 1:(n - 2 - 40) // 32] = -1  # pages that only held tokens outside the window
    cache.k[cache.k.shape[0] - 1] = cache.v[cache.k.shape[0] - 1] = torch.zeros((), device="cuda").to(dtype)
    b_ = fa.flex_kv_cache_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    fa.FLEX_MASK_WINDOW_SINKS, 40, 2)
    assert torch.equal(a[0], b_[0]) and torch.equal(a[1], b_[1])


@pytest.mark.parametrize("dtype", [E4M3, BF16], ids=["e4m3", "bf16"])
def test_attention_not_finite_where_masked(dtype):
    """A token whose value (or key) is not finite: rows that keep it get NaN, rows that do not are untouched."""
    gen = torch.Generator().manual_seed(11)
    lens, Q, page = [100], 5, 16
    cache, table = filled(gen, lens, 1, page, 64, dtype)
    q = torch.randn((1, 3, Q, 64), generator=gen).bfloat16().cuda()
    clean = compare(q, cache, table, lens, page)
    pid, at = int(table[0, 97 // page]), 97 % page       # seen by query tokens 2, 3, 4
    bad = math.nan if dtype == E4M3 else math.inf
    cache.v[pid, 0, at, 7] = torch.tensor(bad, device="cuda").to(dtype)
    out, lse = fa.flex_kv_cache_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert torch.equal(lse, clean[1])
    assert torch.equal(out[:, :, :2], clean[0][:, :, :2])
    hit = torch.zeros(64, dtype=torch.bool, device="cuda")
    hit[7] = True
    assert not out[:, :, 2:, hit].float().isfinite().any()
    assert torch.equal(out[:, :, 2:, ~hit], clean[0][:, :, 2:, ~hit])
    cache.k[pid, 0, at, 0] = torch.tensor(math.nan, device="cuda").to(dtype)
    out, lse = fa.flex_kv_cache_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert torch.equal(out[:, :, :2], clean[0][:, :, :2]) and torch.equal(lse[:, :, :2], clean[1][:, :, :2])
    assert out[:, :, 2:].float().isnan().all() and lse[:, :, 2:].isnan().all()


def test_attention_large_and_small_queries():
    gen = torch.Generator().manual_seed(13)
    lens = [90]
    cache, table = filled(gen, lens, 1, 16, 128, E4M3)
    q = torch.randn((1, 4, 1, 128), generator=gen)
    q[0, 0] *= 1e30
    q[0, 1] *= 1e-30
    q[0, 2] = 0
    q[0, 3, 0, ::2] *= 2.0**-20
    q = q.bfloat16().cuda()
    # scores of the first row scale with it: its softmax is one-hot, lse as large as its scores
    compare(q, cache, table, lens, 16)


def test_attention_beside_a_page_of_large_values():
    """A page whose values (and V scale) are 2^10 times the others', which no query looks at: its share of the
    result is small, and the others keep their bits.  A weight is off by fp16's 2^-11, or by half its smallest step:
    2^-25 in units where the row's largest is 2^7 at least, times the largest V scale and 448."""
    gen = torch.Generator().manual_seed(37)
    lens, page, D, G = [200], 16, 64, 4
    cache, table = filled(gen, lens, 1, page, D, E4M3)
    for i in range(13):
        pid, used = int(table[0, i]), min(page, lens[0] - i * page)
        big = i == 5
        cache.k_scale[pid], cache.v_scale[pid] = 2.0**-6, 2.0**2 if big else 2.0**-8
        k, v = (torch.randn((used, D), generator=gen).cuda() for _ in range(2))
        k[:, 0] = -6.0 if big else 1.0
        for x, y in ((cache.k, k * 64), (cache.v, v * 100)):
            x[pid, 0, :used] = y.clamp(-448, 448).to(E4M3)
    q = torch.randn((1, G, 1, D), generator=gen)
    q[..., 0] = 40.0
    q = q.bfloat16().cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, _ = fa.flex_kv_cache_attention(q, cache, table, n)
    ids = table[0].long()[torch.arange(200, device="cuda") // page]
    k, v = (values(cache, w)[ids, 0, torch.arange(200, device="cuda") % page] for w in "kv")
    s = (q[0, :, 0].double() @ k.T) * D**-0.5
    e_s = 2.0**-24 * (D + 8) * (q[0, :, 0].double().abs() @ k.abs().T).amax(-1, keepdim=True) * D**-0.5
    p = torch.softmax(s, -1)
    total = (s - s.amax(-1, keepdim=True)).exp().sum(-1, keepdim=True)
    want = p @ v
    bound = (2.0**-11 + 2 * e_s + 2.0**-18) * (p @ v.abs()) + 2.0**-32 * 200 * 448 * 4.0 / total + 2.0**-8 * want.abs()
    assert ((out[0, :, 0].double() - want).abs() <= bound).all()


def test_decoding_loop_in_a_graph():
    """Prompt, then steps of rotation + append + attention replayed from one CUDA graph on another stream,
    against attention over the whole sequence with the cache's own rounded values."""
    B, H, G, D, page, steps = 2, 2, 3, 64, 16, 20
    gen = torch.Generator().manual_seed(17)
    prompt = [21, 33]
    table, pages = table_of(gen, [5, 5], 5)
    cache = new_cache(pages, H, page, D, E4M3)
    inv = fa.flex_rope_frequencies(D)
    x = torch.randn((3, B, 33 + steps, H * G, D), generator=gen).bfloat16().cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    fa.flex_kv_cache_append(cache, x[1, :, :33, :H].transpose(1, 2), x[2, :, :33, :H].transpose(1, 2), table, lens, new,
                            inv_freq=inv)
    lens += new
    q, k, v = (torch.empty((B, h, 1, D), dtype=BF16, device="cuda") for h in (H * G, H, H))

    def step():
        qr, _ = fa.flex_rope_fwd(q, None, inv, lens[:, None])
        fa.flex_kv_cache_append(cache, k, v, table, lens, inv_freq=inv)
        lens.add_(1)
        return fa.flex_kv_cache_attention(qr, cache, table, lens, fa.FLEX_MASK_WINDOW_SINKS, 30, 3)

    def put(i):
        for b in range(B):
            for dst, src, h in ((q, 0, H * G), (k, 1, H), (v, 2, H)):
                dst[b, :, 0] = x[src, b, prompt[b] + i, :h]

    put(0)
    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out, lse = step()
    torch.cuda.synchronize()
    for i in range(1, steps):
        put(i)
        graph.replay()
        n = lens.tolist()
        qr, _ = fa.flex_rope_fwd(q, None, inv, (lens - 1)[:, None])
        ro, rl, bo, bl = reference(qr, cache, table, n, page, fa.FLEX_MASK_WINDOW_SINKS, 30, 3, fa.FLEX_SCORE_IDENTITY, 0,
                                   D**-0.5)
        assert ((out.double() - ro).abs() <= bo).all() and ((lse.double() - rl).abs() <= bl).all(), i


def test_other_stream_and_results_repeat():
    gen = torch.Generator().manual_seed(19)
    lens = [700, 300]
    cache, table = filled(gen, lens, 2, 64, 128, E4M3)
    q = torch.randn((2, 8, 1, 128), generator=gen).bfloat16().cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    a = fa.flex_kv_cache_attention(q, cache, table, n)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [fa.flex_kv_cache_attention(q, cache, table, n, stream=s) for s in streams]
    torch.cuda.synchronize()
    for o, l_ in got:
        assert torch.equal(o, a[0]) and torch.equal(l_, a[1])


def test_calls_at_the_same_time():
    """Calls on several streams at once, with the memory that they allocate themselves, and as two graphs."""
    gen = torch.Generator().manual_seed(23)
    lens = torch.randint(2000, 4000, (24,), generator=gen).tolist()
    cache, table = filled(gen, lens, 4, 64, 128, E4M3)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qs = [torch.randn((24, 16, 1, 128), generator=gen).bfloat16().cuda() for _ in range(3)]
    want = [fa.flex_kv_cache_attention(q, cache, table, n) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [fa.flex_kv_cache_attention(qs[0], cache, table, n),
               fa.flex_kv_cache_attention(qs[1], cache, table, n, stream=streams[0]),
               fa.flex_kv_cache_attention(qs[2], cache, table, n, stream=streams[1].cuda_stream)]
        torch.cuda.synchronize()
        for (o, l_), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l_, wl)
    graphs, outs = [], []
    for s, q in zip(streams, qs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append([fa.flex_kv_cache_attention(q, cache, table, n) for _ in range(4)])
        graphs.append(g)
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for results, (wo, wl) in zip(outs, want):
        for o, l_ in results:
            assert torch.equal(o, wo) and torch.equal(l_, wl)


@pytest.mark.parametrize("dtype", [E4M3, BF16], ids=["e4m3", "bf16"])
def test_pages_and_strides_past_32_bits(dtype):
    """Pages behind 2^32 elements of the pool, and new tokens whose strides pass 2^31 elements: as near ones."""
    H, D, page = 4, 128, 256
    pages = 2**32 // (H * page * D) + 6
    gen = torch.Generator().manual_seed(29)
    far, near = fa.flex_kv_cache_create(pages, H, D, page, dtype), new_cache(6, H, page, D, dtype)
    far_table = torch.tensor([[pages - 1, 3], [pages - 4, pages - 2]], dtype=torch.int32, device="cuda")
    near_table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    wide = torch.empty(2**31 + 2**20, dtype=BF16, device="cuda")
    k = wide.as_strided((2, H, 300, D), (2**31, 300 * D, D, 1))
    k.copy_(torch.randn(k.shape, generator=gen).cuda())
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    inv = fa.flex_rope_frequencies(D)
    for cache, table in ((far, far_table), (near, near_table)):
        fa.flex_kv_cache_append(cache, k, k, table, lens, inv_freq=inv)
    for ids, other in zip(far_table.tolist(), near_table.tolist()):
        for i, j, used in zip(ids, other, (page, 300 - page)):
            for x, y in ((far.k, near.k), (far.v, near.v)):
                assert torch.equal(x[i, :, :used].view(torch.uint8), y[j, :, :used].view(torch.uint8))
    q = wide.as_strided((2, 2 * H, 1, D), (2**31, D, D, 1))
    turned = [fa.flex_rope_fwd(x, None, inv)[0] for x in (q, q.contiguous())]
    assert torch.equal(*turned)
    n = torch.tensor([300, 290], dtype=torch.int32, device="cuda")
    a, b = (fa.flex_kv_cache_attention(x, c, t, n) for x, c, t in ((q, far, far_table), (q.contiguous(), near, near_table)))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


FIRST_CALL = """
import torch
from block_sparse_masked_blockmask_gb300 import flexattn as fa
c = fa.flex_kv_cache_create(3, 2, 64, 16, torch.bfloat16)
c.k.normal_(), c.v.normal_()
t = torch.arange(3, dtype=torch.int32, device="cuda")[None]
n = torch.tensor([40], dtype=torch.int32, device="cuda")
q = torch.randn((1, 4, 1, 64), device="cuda").bfloat16()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = fa.flex_kv_cache_attention(q, c, t, n)
g.replay()
want = fa.flex_kv_cache_attention(q, c, t, n)
assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
assert fa.flex_device_status() == fa.FLEX_OK
print("captured")
"""


def test_first_call_of_a_process_is_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
