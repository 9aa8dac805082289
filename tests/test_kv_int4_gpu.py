"""The 4-bit cache as it is written and read back, and packed appends to every kind of cache.

Bounds.  A scale is m / 7 rounded to bf16, whose 8 significant bits make that half of 2^-7: off by 2^-8 of itself at
most; a value lies within half a step (one scale) of what is held.  Both hold for the rotated key, which is off by
2^-20 of its pair's size beforehand (sines, cosines and the float32 sum), and so is m, by the largest of those.  bf16
inputs that are not rotated are held exactly by the rule.
"""
import math

import pytest
import torch

from block_sparse_masked_blockmask_gb300 import flexattn as fa
from test_kv_cache_gpu import rotated, table_of

pytestmark = pytest.mark.gpu
E4M3, BF16, INT4 = torch.float8_e4m3fn, torch.bfloat16, torch.uint8
KINDS = pytest.mark.parametrize("kind", [INT4, E4M3, BF16], ids=["int4", "e4m3", "bf16"])


def order(D):
    """The value that each code of a row stands for, in the order of the row's half bytes."""
    return [32 * j + 4 * g + e for g in range(8) for j in range(D // 32) for e in range(4)]


def codes(held, D):
    """The codes 0 .. 15 of uint8 [..., D / 2], value by value."""
    c = torch.stack((held & 15, held >> 4), -1).flatten(-2).long()
    at = torch.empty(D, dtype=torch.long, device=held.device)
    at[torch.tensor(order(D), device=held.device)] = torch.arange(D, device=held.device)
    return c[..., at]


def values(cache, which):
    """What the cache holds, float64 [pages, H, page, D]."""
    x, s = getattr(cache, which), getattr(cache, which + "_scale")
    D = cache.shape[3]
    if x.dtype == INT4:
        s = s.double()[..., None] if which == "v" else s.double().repeat_interleave(32, -1)
        return (codes(x, D) - 8).double() * s
    return x.double() if s is None else x.double() * s.double()[:, :, None, None]


def new_cache(pages, H, page, D, kind):
    """A cache whose memory holds a pattern that no append writes: codes 0 (or NaN), scales NaN."""
    c = fa.flex_kv_cache_create(pages, H, D, page, kind)
    for x in (c.k, c.v):
        x.copy_(torch.full(x.shape, 0.0 if kind == INT4 else math.nan, device="cuda"))
    if kind != BF16:
        c.k_scale.fill_(math.nan)
        c.v_scale.fill_(math.nan)
    return c


def held_bytes(cache):
    return [x.clone().view(torch.uint8) for x in (cache.k, cache.v, cache.k_scale, cache.v_scale) if x is not None]


def rule(x, group):
    """Codes less 8 and scales of float64 x [..., D]: m / 7 in bf16, halves away from zero."""
    y = x.unflatten(-1, (-1, group))
    m = y.abs().amax(-1)
    s = (m.float() / 7).bfloat16()
    s = torch.where(s.double() < 2.0**-120, torch.zeros_like(s), s)
    q = torch.floor(y.abs() / torch.where(s > 0, s, 1.0).double()[..., None] + 0.5) * torch.sign(y)
    return torch.where(s[..., None] > 0, q, 0.0).flatten(-2).long(), s


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts_of(lens, first=0):
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return ints(at)


@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32], ids=["from_bf16", "from_fp32"])
@pytest.mark.parametrize("page,D,H", [(16, 64, 3), (64, 128, 8), (256, 128, 1), (32, 64, 33)])
def test_append_holds_the_rule(page, D, H, src):
    """Without rotation: every scale and code as the rule has them, ties among them; other slots as they were."""
    gen = torch.Generator().manual_seed(page + D + H)
    calls = [(5, [5, 0, 3, 5]), (1, None), (67, [67, 20, 0, 9]), (1, [1, 1, 0, 1]), (130, [130, 1, 90, 7])]
    width = -(-210 // page)
    table, pages = table_of(gen, [width] * 4, width)
    cache = new_cache(pages, H, page, D, INT4)
    want = held_bytes(cache)
    lens = torch.zeros(4, dtype=torch.int32)
    for n, (S, new) in enumerate(calls):
        k, v = (torch.randn((4, S, H, D), generator=gen).mul(4.0 ** ((n * 3) % 5 - 2)).to(src) for _ in range(2))
        if src == torch.bfloat16:
            # magnitudes of whole and half steps of the scale that a 7 makes: halves go away from zero
            k[:, 0, 0, :] = (torch.arange(D) % 15 - 7).to(src) / 2
            k[:, 0, 0, ::32] = -7.0
            v[:, 0, 0, :] = k[:, 0, 0, :] * 1.25
        k, v = (x.cuda().transpose(1, 2) for x in (k, v))
        fa.flex_kv_cache_append(cache, k, v, table, lens.cuda(), None if new is None else ints(new))
        for b in range(4):
            count = S if new is None else new[b]
            pos = (lens[b] + torch.arange(count)).cuda()
            ids, at = table[b].long()[pos // page], pos % page
            for i, (x, group) in enumerate(((k, 32), (v, D))):
                q, s = rule(x[b, :, :count].double().transpose(0, 1), group)      # [tokens, H, D]
                row = q[..., order(D)].to(torch.uint8) + 8
                want[i][ids, :, at] = row[..., 0::2] | row[..., 1::2] << 4
                s = s if group == 32 else s[..., 0:1]
                want[2 + i].unflatten(-1, (-1, 2)).view(pages, H, page, -1)[ids, :, at] = \
                    s.contiguous().view(torch.uint8)
        lens += S if new is None else torch.tensor(new).int()
        got = held_bytes(cache)
        for name, a, w in zip(("k", "v", "k_scale", "v_scale"), got, want):
            assert torch.equal(a, w), (n, name)


@KINDS
@pytest.mark.parametrize("D,rotary,layout", [(128, 128, fa.FLEX_ROPE_HALF), (128, 64, fa.FLEX_ROPE_HALF),
                                             (128, 48, fa.FLEX_ROPE_HALF), (128, 128, fa.FLEX_ROPE_INTERLEAVED),
                                             (64, 64, fa.FLEX_ROPE_HALF), (64, 16, fa.FLEX_ROPE_HALF),
                                             (64, 48, fa.FLEX_ROPE_INTERLEAVED), (64, 0, fa.FLEX_ROPE_HALF)])
def test_packed_append_as_padded(D, rotary, layout, kind):
    """Packed sequences (some empty, tokens before the first and behind the last) as the padded batch of them."""
    gen = torch.Generator().manual_seed(D + rotary)
    H, page, lens, past = 3, 32, [7, 0, 150, 1, 0, 64, 33], [0, 5, 31, 32, 900, 16, 100]
    width = 8
    table, pages = table_of(gen, [width] * 7, width)
    table[4] = -1
    caches = [new_cache(pages, H, page, D, kind) for _ in range(2)]
    inv = fa.flex_rope_frequencies(rotary, base=500.0) if rotary else None
    k, v = (torch.randn((1, 3 + sum(lens) + 4, H, D), generator=gen).to(BF16).cuda().transpose(1, 2) for _ in range(2))
    starts = starts_of(lens, 3)
    before = held_bytes(caches[0])
    fa.flex_kv_cache_append_packed(caches[0], k, v, starts, table, ints(past), inv, layout, 1.25)
    pk, pv = (torch.full((7, H, max(lens), D), math.nan, dtype=BF16, device="cuda") for _ in range(2))
    for b, n in enumerate(lens):
        at = int(starts[b])
        pk[b, :, :n], pv[b, :, :n] = k[0, :, at:at + n], v[0, :, at:at + n]
    fa.flex_kv_cache_append(caches[1], pk, pv, table, ints(past), ints(lens), inv, layout, 1.25)
    got, want = held_bytes(caches[0]), held_bytes(caches[1])
    for a, w, old in zip(got, want, before):
        assert torch.equal(a, w) and not torch.equal(a, old)
    if kind != INT4 or not rotary:
        return
    # the rotated keys: scales within rounding of m / 7, values within half a step
    scale = caches[0].k_scale.double()
    have = values(caches[0], "k")
    for b, n in enumerate(lens):
        pos = past[b] + torch.arange(n, device="cuda")
        y, size = rotated(k[0, :, int(starts[b]):int(starts[b]) + n], pos, inv, layout)
        y[..., :rotary], size = 1.25 * y[..., :rotary], 1.25 * size * 2.0**-20
        ids, at = table[b].long()[pos // page], pos % page
        s, x = scale[ids, :, at].transpose(0, 1), have[ids, :, at].transpose(0, 1)
        m, e = (t.unflatten(-1, (-1, 32)).abs().amax(-1) for t in (y, size))
        assert ((s - m / 7).abs() <= 2.0**-8 * m / 7 + e).all()
        assert ((x - y).abs() <= 0.5 * s.repeat_interleave(32, -1) * (1 + 2.0**-20) + size).all()


def test_append_odd_values():
    """NaN and infinities (the values that share their scale), zeros, the smallest and the largest magnitudes."""
    H, D, page = 1, 128, 16
    cache = new_cache(1, H, page, D, INT4)
    x = torch.zeros((1, H, 8, D))
    x[0, 0, 1, 40], x[0, 0, 2, 5], x[0, 0, 2, 100] = math.nan, -math.inf, 3.0
    x[0, 0, 3, :] = 2.0**-126
    x[0, 0, 4, ::2] = torch.finfo(torch.float32).max
    x[0, 0, 5, :] = -0.0
    x[0, 0, 6, 0] = 7 * 2.0**-120
    x[0, 0, 7, 0] = 6.9 * 2.0**-120
    fa.flex_kv_cache_append(cache, x.cuda(), x.cuda(), ints([[0]]), ints([0]))
    k, v = values(cache, "k")[0, 0], values(cache, "v")[0, 0]
    nan_k = torch.zeros((8, D), dtype=torch.bool)
    nan_k[1, 32:64] = nan_k[2, 0:32] = True
    assert torch.equal(k[:8].isnan().cpu(), nan_k)
    assert v[1].isnan().all() and v[2].isnan().all() and v[[0, 3, 4, 5, 6, 7]].isfinite().all()
    assert k[2, 100] == codes(cache.k, D)[0, 0, 2, 100].sub(8) * cache.k_scale[0, 0, 2, 3].double()
    assert abs(float(k[2, 100]) - 3.0) <= 3.0 * 2.0**-8
    for y in (k, v):
        assert (y[[0, 3, 5, 7]] == 0).all()
        assert y[6, 0] == 7 * 2.0**-120 and (y[6, 1:] == 0).all()
        top = torch.finfo(torch.float32).max
        assert ((y[4, ::2] - top).abs() <= 2.0**-8 * top).all() and (y[4, 1::2] == 0).all()
    assert (codes(cache.k, D)[0, 0, :8] >= 1).all()


@KINDS
def test_append_drops(kind):
    """Bad pages, tokens past the table, negative lengths; starts that do not ascend touch nothing else's memory."""
    H, D, page = 2, 64, 16
    k = torch.ones((1, H, 120, D), device="cuda").bfloat16()
    table = ints([[-1, 0], [6, 1], [2, -7], [3, 100], [4, 5], [4, 5]])
    lens = ints([0, 0, 0, 30, -1, 40])
    cache = new_cache(6, H, page, D, kind)
    before = held_bytes(cache)[0]
    fa.flex_kv_cache_append_packed(cache, k, k, starts_of([20, 20, 18, 20, 20, 20]), table, lens)
    changed = (held_bytes(cache)[0] != before).any(3).any(1)
    want = torch.zeros((6, page), dtype=torch.bool)
    want[0, :4] = want[1, :4] = want[2, :] = True
    assert torch.equal(changed.cpu(), want)
    fa.flex_kv_cache_append_packed(cache, k, k, ints([50, 10, 300, -5, 20, 7, 90]), table.clamp(0, 5), ints([0] * 6))
    fa.flex_kv_cache_read(cache, table, ints([50, 10, 300, -5, 20, 7, 90]), 100)
    torch.cuda.synchronize()


@KINDS
def test_starts_far_below_zero(kind):
    """Starts whose distance from a token passes 32 bits: positions that no table has."""
    H, D, page, low = 2, 64, 16, -2**31
    k = torch.ones((1, H, 120, D), device="cuda").bfloat16()
    table, lens = ints([[0, 1], [2, 3]]), ints([0, 31])
    cache = new_cache(4, H, page, D, kind)
    before = held_bytes(cache)
    for starts in ([low, 120, 120], [low, low + 5, 120]):
        fa.flex_kv_cache_append_packed(cache, k, k, ints(starts), table, lens)
        for x in fa.flex_kv_cache_read(cache, table, ints(starts), 120):
            assert (x == 0).all()
    assert all(torch.equal(x, y) for x, y in zip(held_bytes(cache), before))


@KINDS
@pytest.mark.parametrize("B", [127, 128, 300])
def test_many_sequences(B, kind):
    """As many as a CTA keeps the starts of, and more: packed against padded appends, and what is read back."""
    gen = torch.Generator().manual_seed(B)
    H, D, page = 2, 64, 16
    lens = torch.randint(0, 4, (B,), generator=gen).tolist()
    table, pages = table_of(gen, [1] * B, 1)
    starts, zero = starts_of(lens), ints([0] * B)
    k, v = (torch.randn((1, H, sum(lens), D), generator=gen).to(BF16).cuda() for _ in range(2))
    one, other = (new_cache(pages, H, page, D, kind) for _ in range(2))
    fa.flex_kv_cache_append_packed(one, k, v, starts, table, zero)
    padded = [torch.zeros((B, H, 3, D), dtype=BF16, device="cuda") for _ in range(2)]
    for x, y in zip(padded, (k, v)):
        for b, n in enumerate(lens):
            x[b, :, :n] = y[0, :, int(starts[b]):int(starts[b]) + n]
    fa.flex_kv_cache_append(other, *padded, table, zero, ints(lens))
    assert all(torch.equal(x, y) for x, y in zip(held_bytes(one), held_bytes(other)))
    for w, x in zip("kv", fa.flex_kv_cache_read(one, table, starts, sum(lens), dtype=torch.float32)):
        held = values(one, w)
        for b, n in enumerate(lens):
            assert torch.equal(x[0, :, int(starts[b]):int(starts[b]) + n], held[int(table[b, 0]), :, :n].float())


@KINDS
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["to_bf16", "to_fp32"])
@pytest.mark.parametrize("D,page,H", [(64, 16, 1), (128, 64, 8), (128, 256, 3), (64, 32, 17)])
def test_read(D, page, H, out, kind):
    """Every value of a cache of random bits, ragged; positions without a page, tokens outside of the sequences."""
    gen = torch.Generator().manual_seed(D + page)
    lens = [1, 0, 300, 17, 64, 0, 129]
    counts = [-(-n // page) for n in lens]
    width = max(counts) + 1
    table, pages = table_of(gen, counts, width)
    c = fa.flex_kv_cache_create(pages, H, D, page, kind)
    for x in (c.k, c.v):
        if kind == INT4:
            x.copy_(torch.randint(0, 256, x.shape, generator=gen))
        else:
            x.copy_((torch.randn(x.shape, generator=gen) * 50).clamp(-448, 448))
    if kind != BF16:
        for s in (c.k_scale, c.v_scale):
            s.copy_(torch.rand(s.shape, generator=gen) + 0.01)
    bad = (2, 1) if counts[2] > 1 else (2, 0)
    table[bad] = -3
    starts, total = starts_of(lens, 2), 2 + sum(lens) + 5
    kv = [torch.full((1, total, H, D + 8), 77.0, dtype=out, device="cuda")[..., :D].transpose(1, 2) for _ in range(2)]
    got = fa.flex_kv_cache_read(c, table, starts, k_out=kv[0], v_out=kv[1])
    fresh = fa.flex_kv_cache_read(c, table, starts, total, dtype=out)
    for w, x, y in zip("kv", got, fresh):
        held = values(c, w).float()   # exact: 4 bits times 8 or 24 rounded once
        if kind == E4M3:
            held = getattr(c, w).float() * getattr(c, w + "_scale")[:, :, None, None]
        want = torch.full((1, H, total, D), 77.0, dtype=out, device="cuda")
        for b, n in enumerate(lens):
            pos = torch.arange(n, device="cuda")
            ids = table[b].long()[pos // page]
            rows = held[ids.clamp(min=0), :, pos % page] * (ids >= 0)[:, None, None]
            want[0, :, int(starts[b]):int(starts[b]) + n] = rows.transpose(0, 1).to(out)
        assert torch.equal(x, want), w
        inside = slice(int(starts[0]), int(starts[-1]))
        assert torch.equal(y[:, :, inside], want[:, :, inside]), w


@KINDS
def test_write_and_read_on_another_stream_and_captured(kind):
    """The pair replayed from a graph with new inputs each time, beside the same on two more streams."""
    gen = torch.Generator().manual_seed(3)
    H, D, page, lens, past = 2, 128, 16, [40, 3, 17], [5, 0, 30]
    table, pages = table_of(gen, [5, 1, 4], 5)
    inv = fa.flex_rope_frequencies(64)
    starts, every = starts_of(lens), starts_of([n + p for n, p in zip(lens, past)])
    x = torch.randn((4, 2, 1, sum(lens), H, D), generator=gen).to(BF16).cuda()
    k, v = (x[0, i].clone().transpose(1, 2) for i in range(2))

    def fresh():
        c = new_cache(pages, H, page, D, kind)
        fa.flex_kv_cache_append_packed(c, torch.ones((1, H, sum(past), D), dtype=BF16, device="cuda"),
                                       torch.ones((1, H, sum(past), D), dtype=BF16, device="cuda"), starts_of(past), table,
                                       ints([0, 0, 0]))
        return c

    def pair(c, stream=None):
        fa.flex_kv_cache_append_packed(c, k, v, starts, table, ints_past, inv, stream=stream)
        return fa.flex_kv_cache_read(c, table, every, sum(lens) + sum(past), stream=stream)

    ints_past = ints(past)
    cache = fresh()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = pair(cache)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(4):
        k.copy_(x[i, 0].transpose(1, 2)), v.copy_(x[i, 1].transpose(1, 2))
        others = [fresh() for _ in range(3)]
        want = pair(others[0])
        torch.cuda.synchronize()
        graph.replay()
        got = [pair(c, s) for c, s in zip(others[1:], (streams[0], streams[1].cuda_stream))]
        torch.cuda.synchronize()
        if kind == E4M3 and i:   # a page's scale only grows: replays on one cache keep the largest
            continue
        for o in [out] + got:
            assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1]), i


@KINDS
def test_far_pages_and_strides(kind):
    """Pages behind 2^32 values of the pool, and packed tokens whose strides pass 2^31 elements."""
    H, D, page, gen = 4, 128, 256, torch.Generator().manual_seed(5)
    pages = 2**32 // (H * page * D) + 6
    far, near = fa.flex_kv_cache_create(pages, H, D, page, kind), new_cache(6, H, page, D, kind)
    far_table, near_table = ints([[pages - 1, 3], [pages - 4, pages - 2]]), ints([[0, 1], [2, 3]])
    wide = torch.empty(2**31 + 2**27, dtype=BF16, device="cuda")
    k = wide.as_strided((1, 4, 500, D), (2**31, 2**29 + 2**24, D, 1))
    k.copy_(torch.randn(k.shape, generator=gen).cuda())
    starts, lens = starts_of([290, 210]), ints([0, 0])
    inv = fa.flex_rope_frequencies(D)
    outs = []
    for cache, table in ((far, far_table), (near, near_table)):
        fa.flex_kv_cache_append_packed(cache, k, k, starts, table, lens, inv)
        outs.append(fa.flex_kv_cache_read(cache, table, starts, 500))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert outs[0][1].isfinite().all()
