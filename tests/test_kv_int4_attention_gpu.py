"""Attention against the 4-bit cache: the formula in float64 over the values that the cache holds.

Bounds.  A score is a float32 sum of D exact products, group by group, each group's times its scale: off by at most
(D + 16) 2^-24 scale sum |q k|; a query value below 2^-14 of its row's largest keeps fp16's smallest step, 2^-24 of
that one, half of it off.  lse is off by as much, plus 2^-19 for exponentials and sums.  A weight times its value's scale
is rounded to fp16: off by 2^-11 of itself, or by half of fp16's smallest step, 2^-25, in units in which the row's
largest is at least 2^7 (scales below 2^-60 count as 2^-60 there); codes are 8 at most.  The sums of codes (up to 15)
and of the 8 that is taken off afterwards are float32 sums over steps of 16 tokens, each of which cuts off less than
2^-22 of what is summed, and products of numbers that keep 4 of 11 bits, cut off 2^-24 below what 11 bits would make, 2^-17
of the largest, twice: 2^-16 + (n / 16 + 2) 2^-22 times 24 times the sum of weights and scales.  out is rounded once, 2^-8.
That bound is of the worst case, and loose for long sequences: all rows together are off by 2^-8 / sqrt(3) (2-norm) of the
last rounding, 2^-11 of the weights'.
"""
import math

import pytest
import torch

from block_sparse_masked_blockmask_gb300 import flexattn as fa
from test_kv_cache_gpu import MASKS, table_of
from test_kv_int4_gpu import codes, ints, starts_of, values

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def filled(gen, lens, H, page, D, spread=6, extra_width=2):
    """A cache of random codes for these lengths, scales 2^spread apart; scales of free slots are NaN."""
    counts = [-(-n // page) for n in lens]
    width = max(1, max(counts)) + extra_width
    table, pages = table_of(gen, counts, width)
    c = fa.flex_kv_cache_create(pages, H, D, page, torch.uint8)
    for x in (c.k, c.v):
        x.copy_(torch.randint(0, 256, x.shape, generator=gen))
    c.k_scale.fill_(math.nan), c.v_scale.fill_(math.nan)
    for b, n in enumerate(lens):
        for i in range(counts[b]):
            used, pid = min(page, n - i * page), int(table[b, i])
            for s, size in ((c.k_scale, 0.25), (c.v_scale, 1.0)):
                shape = s[pid, :, :used].shape
                s[pid, :, :used] = (size * (1 + torch.rand(shape, generator=gen)) *
                                    2.0 ** -torch.randint(0, spread + 1, shape, generator=gen)).cuda().to(BF16)
    return c, table


def reference(q, cache, table, lens, kind, window, sinks, score, cap, scale):
    """float64 out, lse, and bounds of both."""
    B, Hq, Q, D = q.shape
    P, H, page, _ = cache.shape
    G = Hq // H
    out = torch.zeros((B, Hq, Q, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Q), -math.inf, dtype=torch.float64, device="cuda")
    bo, bl = torch.zeros_like(out), torch.zeros_like(lse)
    kd, vd = values(cache, "k"), values(cache, "v")
    slope = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float64) / Hq)
    for b, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        ids = table[b].long()[at // page]
        good = (ids >= 0) & (ids < P)
        ids = ids.clamp(0, P - 1)
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
            small = qt.abs().amax(-1)[..., None] * k.abs().sum(-1)[:, None] * abs(scale) * 2.0**-25
            if score == fa.FLEX_SCORE_SOFTCAP:
                s = cap * torch.tanh(s / cap)
            elif score == fa.FLEX_SCORE_ALIBI:
                far = slope.reshape(H, G, 1) * (pos - idx).double()
                s, size = s - far, size + far.abs()
            p = torch.softmax(s, -1)
            lse[b, :, t] = torch.logsumexp(s, -1).reshape(-1)
            out[b, :, t] = torch.einsum("hgn,hnd->hgd", p, v).reshape(Hq, D)
            e_s = ((D + 16) * 2.0**-24 * size + small).amax(-1).reshape(-1)
            bl[b, :, t] = e_s + 2.0**-19 * (1 + lse[b, :, t].abs())
            absolute = torch.einsum("hgn,hnd->hgd", p, v.abs()).reshape(Hq, D)
            ref = cache.v_scale[ids[idx], :, idx % page].double().clamp(min=2.0**-60).t()        # [H, n]
            least = 2.0**-32 * 8 * len(idx) * (p * ref[:, None]).amax(-1).reshape(-1)
            sums = (2.0**-16 + (len(idx) / 16 + 2) * 2.0**-22) * 24 * (p * ref[:, None]).sum(-1).reshape(-1)
            bo[b, :, t] = (2.0**-11 + 2 * e_s[:, None] + 2.0**-18) * absolute + 2.0**-8 * out[b, :, t].abs() + \
                (least + sums)[:, None]
    return out, lse, bo, bl


def compare(q, cache, table, lens, kind=fa.FLEX_MASK_CAUSAL, window=0, sinks=0, score=fa.FLEX_SCORE_IDENTITY, cap=5.0,
            scale=None):
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
    out, lse = fa.flex_kv_cache_attention(q, cache, table, ints(lens), kind, window, sinks, score, cap, scale)
    ro, rl, bo, bl = reference(q, cache, table, lens, kind, window, sinks, score, cap, scale)
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(lse), empty) and (out[empty] == 0).all()
    off = torch.where(empty, 0.0, lse.double() - rl).abs()
    assert (off <= bl).all(), float((off - bl).max())
    diff = (out.double() - ro).abs()
    assert (diff <= bo).all(), float((diff - bo).max())
    if ro.count_nonzero() >= 4096 and abs(scale) * float(q.abs().max()) < 1.0:
        assert float(diff.norm()) <= (2.0**-8 / math.sqrt(3) + 2.0**-11) * float(ro.norm())
    return out, lse


@pytest.mark.parametrize("D,page", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 256)])
@pytest.mark.parametrize("H,G,Q", [(1, 1, 1), (2, 4, 1), (1, 8, 2), (2, 3, 5), (1, 1, 9), (1, 17, 1), (1, 5, 7)])
def test_attention(H, G, Q, D, page):
    lens = [1, 0, 17, 130, 300, 64, 3]
    gen = torch.Generator().manual_seed(D + page + 7 * H * G * Q)
    cache, table = filled(gen, lens, H, page, D)
    q = torch.randn((len(lens), Q, H * G, D), generator=gen).to(BF16).cuda().transpose(1, 2)
    scores = (fa.FLEX_SCORE_IDENTITY, fa.FLEX_SCORE_SOFTCAP, fa.FLEX_SCORE_ALIBI)
    for i, (kind, window, sinks) in enumerate(MASKS):
        compare(q, cache, table, lens, kind, window, sinks, scores[i % 3])


@pytest.mark.parametrize("lens,G,Q", [([20000], 8, 1), ([3000, 1, 2999], 2, 1), ([5000], 4, 33)])
def test_attention_long(lens, G, Q):
    gen = torch.Generator().manual_seed(lens[0])
    cache, table = filled(gen, lens, 2, 64, 128)
    q = torch.randn((len(lens), 2 * G, Q, 128), generator=gen).to(BF16).cuda()
    compare(q, cache, table, lens)
    compare(q, cache, table, lens, fa.FLEX_MASK_WINDOW_SINKS, 1000, 5, fa.FLEX_SCORE_ALIBI)


@pytest.mark.parametrize("D,G,Q", [(128, 4, 1), (128, 1, 1), (64, 8, 1), (64, 2, 2), (128, 4, 3), (64, 16, 1)])
def test_attention_many_steps(D, G, Q):
    """A ragged batch large enough that every warp of the launch walks over many steps, sequences and heads."""
    gen = torch.Generator().manual_seed(D + G)
    lens = torch.randint(1, 9000, (40,), generator=gen).tolist()
    lens[3], lens[4], lens[20] = 0, 1, 9000
    cache, table = filled(gen, lens, 8, 64, D)
    q = torch.randn((40, 8 * G, Q, D), generator=gen).to(BF16).cuda()
    compare(q, cache, table, lens)


@pytest.mark.parametrize("B", [129, 1000])
def test_attention_many_sequences(B):
    gen = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 90, (B,), generator=gen).tolist()
    cache, table = filled(gen, lens, 2, 32, 64)
    q = torch.randn((B, 4, 2, 64), generator=gen).to(BF16).cuda()
    compare(q, cache, table, lens)
    compare(q, cache, table, lens, fa.FLEX_MASK_WINDOW_SINKS, 10, 3)


def test_attention_shared_and_bad_pages():
    """Two sequences on the same pages; entries that name no page are masked; entries behind a window are not read."""
    gen = torch.Generator().manual_seed(9)
    lens = [200, 150, 180]
    cache, table = filled(gen, lens, 2, 32, 64)
    table[1, :5] = table[0, :5]
    table[2, 1], table[2, 3] = -1, cache.shape[0]
    q = torch.randn((3, 4, 2, 64), generator=gen).to(BF16).cuda()
    compare(q, cache, table, lens)
    a = compare(q, cache, table, lens, fa.FLEX_MASK_WINDOW_SINKS, 40, 2)
    for b, n in enumerate(lens):
        table[b, 1:(n - 2 - 40) // 32] = -1  # pages that only held tokens outside the window
    b_ = fa.flex_kv_cache_attention(q, cache, table, ints(lens), fa.FLEX_MASK_WINDOW_SINKS, 40, 2)
    assert torch.equal(a[0], b_[0]) and torch.equal(a[1], b_[1])


@pytest.mark.parametrize("at", [97, 30])
def test_attention_not_finite_where_masked(at):
    """A token whose scale is NaN (values, then keys): rows that keep it get NaN, rows that do not are untouched."""
    gen = torch.Generator().manual_seed(11)
    lens, Q, page, window = [100], 5, 16, 67
    cache, table = filled(gen, lens, 1, page, 64)
    q = torch.randn((1, 3, Q, 64), generator=gen).to(BF16).cuda()
    kind = fa.FLEX_MASK_SLIDING_WINDOW
    clean = compare(q, cache, table, lens, kind, window)
    pid, slot = int(table[0, at // page]), at % page
    keep = torch.tensor([p - window < at <= p for p in range(95, 100)], device="cuda")
    assert keep.any() and not keep.all()
    cache.v_scale[pid, 0, slot] = math.nan
    out, lse = fa.flex_kv_cache_attention(q, cache, table, ints(lens), kind, window)
    assert torch.equal(lse, clean[1]) and torch.equal(out[:, :, ~keep], clean[0][:, :, ~keep])
    assert out[:, :, keep].isnan().all()
    cache.k_scale[pid, 0, slot, 1] = math.nan
    out, lse = fa.flex_kv_cache_attention(q, cache, table, ints(lens), kind, window)
    assert torch.equal(out[:, :, ~keep], clean[0][:, :, ~keep]) and torch.equal(lse[:, :, ~keep], clean[1][:, :, ~keep])
    assert out[:, :, keep].isnan().all() and lse[:, :, keep].isnan().all()


def test_attention_large_and_small_queries():
    gen = torch.Generator().manual_seed(13)
    lens = [90]
    cache, table = filled(gen, lens, 1, 16, 128)
    q = torch.randn((1, 4, 1, 128), generator=gen)
    q[0, 0] *= 1e30
    q[0, 1] *= 1e-30
    q[0, 2] = 0
    q[0, 3, 0, ::2] *= 2.0**-20
    compare(q.to(BF16).cuda(), cache, table, lens)


@pytest.mark.parametrize("power", [-112, -114, -120, -126, -133, 100])
def test_attention_queries_at_the_ends_of_the_type(power):
    """Rows of 2^power times small whole numbers (exact down to bf16's smallest step), with scales that bring scores back."""
    gen = torch.Generator().manual_seed(300 + power)
    cache, table = filled(gen, [70, 33], 1, 32, 64)
    q = (torch.randint(-7, 8, (2, 4, 1, 64), generator=gen).double() * 2.0**power).to(BF16).cuda()
    q[1, 3] = 0
    assert (q[0] != 0).any()
    for scale in (0.125, 2.0**min(-power - 6, 100)):
        compare(q, cache, table, [70, 33], scale=scale)


@pytest.mark.parametrize("D,G", [(64, 4), (128, 12)])
@pytest.mark.parametrize("spread", [40, 100])
def test_attention_scales_far_apart(D, G, spread):
    """Values whose scales are 2^spread apart, the large ones where a row hardly looks, or tokens of small ones alone."""
    gen = torch.Generator().manual_seed(spread + G)
    lens, page = [400, 70], 16
    cache, table = filled(gen, lens, 1, page, D, spread=0)
    cache.v_scale.mul_(2.0 ** torch.randint(-spread // 2, spread // 2 + 1, cache.v_scale.shape, generator=gen).cuda())
    q = torch.randn((2, G, 1, D), generator=gen).to(BF16).cuda() * 4
    compare(q, cache, table, lens)
    # first tokens of large values that score far below: the others' bits count where those have next to no weight
    ids = table[0].long()[torch.arange(64, device="cuda") // page]
    cache.v_scale[ids, :, torch.arange(64, device="cuda") % page] = 2.0**(spread // 2)
    compare(q, cache, table, lens, score=fa.FLEX_SCORE_ALIBI)
    # zeros: a value that stands for nothing, however much weight it has
    cache.v_scale[int(table[1, 0])] = 0.0
    compare(q, cache, table, lens)
    cache.v_scale[table[1, :5].long().clamp(min=0)] = 0.0
    out, lse = fa.flex_kv_cache_attention(q, cache, table, ints(lens))
    assert (out[1] == 0).all() and lse.isfinite().all()


def test_calls_at_the_same_time_and_repeated():
    """Calls on several streams at once and as graphs, with memory that they allocate themselves: the same bits."""
    gen = torch.Generator().manual_seed(23)
    lens = torch.randint(2000, 4000, (24,), generator=gen).tolist()
    cache, table = filled(gen, lens, 4, 64, 128)
    n = ints(lens)
    qs = [torch.randn((24, 16, 1, 128), generator=gen).to(BF16).cuda() for _ in range(3)]
    want = [fa.flex_kv_cache_attention(q, cache, table, n) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
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
    assert fa.flex_device_status() == fa.FLEX_OK


def test_far_pages():
    """Pages whose codes lie behind 2^32 bytes of the pool, against the same contents on near pages."""
    H, D, page = 4, 128, 256
    pages, gen = 2**32 // (H * page * D // 2) + 6, torch.Generator().manual_seed(29)
    far, near = (fa.flex_kv_cache_create(n, H, D, page, torch.uint8) for n in (pages, 4))
    far_table, near_table = ints([[pages - 1, 3], [pages - 4, pages - 2]]), ints([[0, 1], [2, 3]])
    k, v = (torch.randn((2, H, 300, D), generator=gen).to(BF16).cuda() for _ in range(2))
    lens, q = ints([300, 290]), torch.randn((2, 2 * H, 1, D), generator=gen).to(BF16).cuda()
    got = []
    for cache, table in ((far, far_table), (near, near_table)):
        fa.flex_kv_cache_append(cache, k, v, table, ints([0, 0]))
        got.append(fa.flex_kv_cache_attention(q, cache, table, lens))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert got[0][0].isfinite().all()


def test_decoding_in_a_graph():
    """Packed prompts, then steps of rotation + append + attention replayed from one CUDA graph, against attention over
    the whole sequence with the values that the cache holds."""
    B, H, G, D, page, steps = 3, 2, 3, 64, 16, 20
    gen = torch.Generator().manual_seed(17)
    prompt = [21, 0, 33]
    table, pages = table_of(gen, [4, 2, 5], 5)
    cache = fa.flex_kv_cache_create(pages, H, D, page, torch.uint8)
    cache.k_scale.fill_(math.nan), cache.v_scale.fill_(math.nan)
    inv = fa.flex_rope_frequencies(D)
    first = torch.randn((2, 1, sum(prompt), H, D), generator=gen).to(BF16).cuda().transpose(2, 3)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    fa.flex_kv_cache_append_packed(cache, first[0], first[1], starts_of(prompt), table, lens, inv)
    lens += ints(prompt)
    x = torch.randn((steps, B, 1, H * (G + 2), D), generator=gen).to(BF16).cuda()
    now = x[0].clone()
    q, k, v = (y.transpose(1, 2) for y in now.split([H * G, H, H], 2))

    def step():
        qr, _ = fa.flex_rope_fwd(q, None, inv, lens[:, None])
        fa.flex_kv_cache_append(cache, k, v, table, lens, inv_freq=inv)
        lens.add_(1)
        return fa.flex_kv_cache_attention(qr, cache, table, lens, fa.FLEX_MASK_WINDOW_SINKS, 30, 3)

    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out, lse = step()
    torch.cuda.synchronize()
    for i in range(1, steps):
        now.copy_(x[i])
        graph.replay()
        qr, _ = fa.flex_rope_fwd(q, None, inv, (lens - 1)[:, None])
        ro, rl, bo, bl = reference(qr, cache, table, lens.tolist(), fa.FLEX_MASK_WINDOW_SINKS, 30, 3, fa.FLEX_SCORE_IDENTITY,
                                   0, D**-0.5)
        assert ((out.double() - ro).abs() <= bo).all() and ((lse.double() - rl).abs() <= bl).all(), i
    assert codes(cache.k, D).amin() >= 0
