"""Attention over packed sequences with grouped query heads: the formula in float64, sequence by sequence.

Bounds.  A score is a float32 sum of D exact products: off by at most (D + 8) 2^-24 scale sum |q k|, and what ALiBi and the
softcap add is off by 2^-22 of its terms; so is lse, plus 2^-19 for exponentials and sums.  Weights are rounded to bf16
(2^-8), the row's sum is not; out is rounded once more (2^-8).
"""
import math
import os
import subprocess
import sys

import pytest
import torch

from block_sparse_masked_blockmask_gb300 import flexattn as fa
from test_kv_cache_gpu import table_of
from test_kv_int4_gpu import ints, starts_of

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
MASKS = [(fa.FLEX_MASK_CAUSAL, 0, 0), (fa.FLEX_MASK_SLIDING_WINDOW, 5, 0), (fa.FLEX_MASK_SLIDING_WINDOW, 0, 0),
         (fa.FLEX_MASK_SLIDING_WINDOW, 200, 0), (fa.FLEX_MASK_WINDOW_SINKS, 33, 4), (fa.FLEX_MASK_WINDOW_SINKS, 1, 170),
         (fa.FLEX_MASK_WINDOW_SINKS, 0, 3), (fa.FLEX_MASK_WINDOW_SINKS, 2**31 - 1, 2**31 - 1),
         (fa.FLEX_MASK_WINDOW_SINKS, 130, 129), (fa.FLEX_MASK_ALL, 0, 0), (fa.FLEX_MASK_WINDOW_SINKS, 300, 20)]
SCORES = (fa.FLEX_SCORE_IDENTITY, fa.FLEX_SCORE_SOFTCAP, fa.FLEX_SCORE_ALIBI)


def row_keep(pos, kv, kind, window, sinks):
    if kind == fa.FLEX_MASK_ALL:
        return torch.ones((len(pos), len(kv)), dtype=torch.bool, device=kv.device)
    far = pos[:, None] - kv
    keep = far >= 0
    if kind != fa.FLEX_MASK_CAUSAL:
        keep &= (far < window) | (kv < (sinks if kind == fa.FLEX_MASK_WINDOW_SINKS else 0))
    return keep


def reference(q, k, v, qs, ks, kind, window, sinks, score, cap, scale):
    """float64 out, lse and their bounds [Hq, T, D] and [Hq, T]; NaN where no sequence has a row."""
    q, k, v = q[0].double(), k[0].double(), v[0].double()
    Hq, T, D = q.shape
    G = Hq // k.shape[0]
    out, bo = torch.full_like(q, math.nan), torch.zeros_like(q)
    lse, bl = torch.full((Hq, T), math.nan, dtype=torch.float64, device="cuda"), torch.zeros((Hq, T), device="cuda").double()
    slope = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float64) / Hq)
    for qa, qe, ka, ke in zip(qs[:-1], qs[1:], ks[:-1], ks[1:]):
        n, m = qe - qa, ke - ka
        if n == 0:
            continue
        pos, kv = torch.arange(m - n, m, device="cuda"), torch.arange(m, device="cuda")
        keep = row_keep(pos, kv, kind, window, sinks)
        for h in range(Hq):
            kh, vh = k[h // G, ka:ke], v[h // G, ka:ke]
            s = q[h, qa:qe] @ kh.T * scale
            size = q[h, qa:qe].abs() @ kh.abs().T * abs(scale)
            err = (D + 8) * 2.0**-24 * size
            if score == fa.FLEX_SCORE_SOFTCAP:
                s = cap * torch.tanh(s / cap)
                err = err + 2.0**-22 * s.abs()
            elif score == fa.FLEX_SCORE_ALIBI:
                far = slope[h] * (pos[:, None] - kv).double()
                s, err = s - far, err + 2.0**-22 * far.abs()
            s = s.masked_fill(~keep, -math.inf)
            live = keep.any(1)
            p = torch.where(live[:, None], torch.softmax(s, -1), 0.0).nan_to_num(0.0) if m else torch.zeros_like(s)
            lse[h, qa:qe] = torch.logsumexp(s, -1) if m else -math.inf
            # a key's error counts by what weight it has, and a little of itself
            e_s = ((p + 2.0**-12) * err.masked_fill(~keep, 0.0)).amax(-1) * 2 + (p * err.masked_fill(~keep, 0.0)).sum(-1) \
                if m else torch.zeros(n, device="cuda").double()
            bl[h, qa:qe] = e_s + 2.0**-19 * (1 + lse[h, qa:qe].nan_to_num(neginf=0.0).abs())
            out[h, qa:qe] = p @ vh
            bo[h, qa:qe] = (2.0**-8 + 2 * e_s[:, None] + 2.0**-18) * (p @ vh.abs()) + 2.0**-8 * out[h, qa:qe].abs()
    return out, lse, bo, bl


def tokens(gen, total, heads, D, order, size=1.0):
    if order == "thd":
        return (torch.randn((1, total, heads, D), generator=gen) * size).to(BF16).cuda().transpose(1, 2)
    return (torch.randn((1, heads, total, D), generator=gen) * size).to(BF16).cuda()


def compare(q, k, v, qs, ks, kind=fa.FLEX_MASK_CAUSAL, window=0, sinks=0, score=fa.FLEX_SCORE_IDENTITY, cap=3.0, scale=None,
            out=None, plan=None):
    scale = q.shape[3] ** -0.5 if scale is None else scale
    if plan is None:
        plan = fa.flex_packed_plan_create(ints(qs), ints(ks), q.shape[2], k.shape[2], q.shape[1], k.shape[1], kind, window,
                                          sinks)
    lse = torch.full(q.shape[:3], 77.0, device="cuda")
    out = torch.full(q.shape, 77.0, dtype=BF16, device="cuda") if out is None else out
    got = fa.flex_attention_packed_fwd(q, k, v, plan, score, cap, scale, out=out, lse=lse)
    assert got[0] is out and fa.flex_device_status() == fa.FLEX_OK
    ro, rl, bo, bl = reference(q, k, v, qs, ks, kind, window, sinks, score, cap, scale)
    o, l_ = out[0].double(), lse[0].double()
    none = rl.isnan()                                   # tokens outside of the sequences: as they were
    assert (o[none] == 77).all() and (l_[none] == 77).all()
    empty = torch.isneginf(rl)
    assert torch.equal(torch.isneginf(l_), empty) and (o[empty] == 0).all()
    off = torch.where(empty | none, 0.0, l_ - rl).abs()
    assert (off <= bl).all(), (float((off - bl).max()), float(off.max()))
    diff = torch.where(none[..., None], 0.0, o - ro).abs()
    assert (diff <= bo).all(), (float((diff - bo).max()), float(diff.max()))
    return out, lse


def running(lens, first=0):
    return starts_of(lens, first).tolist()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hk,G,order", [(1, 1, "htd"), (2, 4, "thd"), (3, 2, "thd"), (1, 5, "thd"), (2, 8, "htd"), (1, 16, "thd"),
                                        (1, 3, "htd"), (1, 32, "thd")])
def test_masks_and_lengths(D, Hk, G, order):
    """Ragged prompts (empty, one token, tile ends) at every mask and score; tokens before and behind all of them."""
    gen = torch.Generator().manual_seed(D + 10 * G)
    for lens in ([5, 0, 1, 128, 300, 127, 129, 2, 33], [700, 1, 384]):  # few kv tiles a sequence, and more
        qs = running(lens, 3)
        q = tokens(gen, qs[-1] + 9, Hk * G, D, order)
        k, v = (tokens(gen, qs[-1] + 9, Hk, D, order) for _ in range(2))
        for i, (kind, window, sinks) in enumerate(MASKS):
            compare(q, k, v, qs, qs, kind, window, sinks, SCORES[i % 3])


@pytest.mark.parametrize("D,Hk,G", [(64, 2, 4), (128, 1, 6), (128, 2, 1), (64, 1, 20)])
def test_earlier_keys(D, Hk, G):
    """Parts of prompts behind earlier keys, and fewer keys than queries (rows at negative positions), or none."""
    gen = torch.Generator().manual_seed(D + G)
    new, keys = [40, 1, 0, 200, 17, 130, 64, 300, 9], [700, 129, 50, 200, 3, 0, 1000, 131, 0]
    qs, ks = running(new), running(keys, 2)
    q = tokens(gen, qs[-1], Hk * G, D, "thd")
    k, v = (tokens(gen, ks[-1] + 1, Hk, D, "thd") for _ in range(2))
    for i, (kind, window, sinks) in enumerate(MASKS):
        compare(q, k, v, qs, ks, kind, window, sinks, SCORES[(i + 1) % 3])


@pytest.mark.parametrize("D,Hk,G,lens", [(128, 2, 4, [3001]), (64, 1, 8, [2500, 10, 1700]), (128, 8, 4, [700, 650, 3, 512])])
def test_long_prompts(D, Hk, G, lens):
    """More items than SMs, so that CTAs take several of them."""
    gen = torch.Generator().manual_seed(sum(lens))
    qs = running(lens)
    q = tokens(gen, qs[-1], Hk * G, D, "thd")
    k, v = (tokens(gen, qs[-1], Hk, D, "thd") for _ in range(2))
    compare(q, k, v, qs, qs)
    compare(q, k, v, qs, qs, fa.FLEX_MASK_WINDOW_SINKS, 400, 130, fa.FLEX_SCORE_ALIBI)


def test_many_sequences():
    gen = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 40, (700,), generator=gen).tolist()
    qs = running(lens)
    q, k, v = tokens(gen, qs[-1], 8, 64, "thd"), tokens(gen, qs[-1], 2, 64, "thd"), tokens(gen, qs[-1], 2, 64, "thd")
    compare(q, k, v, qs, qs)


@pytest.mark.parametrize("score,cap", [(fa.FLEX_SCORE_SOFTCAP, 0.01), (fa.FLEX_SCORE_SOFTCAP, 1e6), (fa.FLEX_SCORE_IDENTITY, 1)])
def test_large_scores(score, cap):
    """Scores of hundreds, rising along the keys, so that the running maximum is raised again and again."""
    gen = torch.Generator().manual_seed(2)
    qs = running([600, 90])
    q, k, v = tokens(gen, 690, 4, 128, "thd", 6.0), tokens(gen, 690, 1, 128, "thd", 6.0), tokens(gen, 690, 1, 128, "thd")
    k *= (torch.arange(690, device="cuda") % 200 / 100.0).to(BF16)[:, None]
    compare(q, k, v, qs, qs, score=score, cap=cap)


@pytest.mark.parametrize("D,G", [(64, 4), (128, 4), (128, 1), (64, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 2)])
@pytest.mark.parametrize("at,last", [(10, 50), (200, 50), (259, 50), (10, 1500), (200, 1500), (259, 1500)])
def test_not_finite_where_masked(D, G, window, sinks, at, last):
    """A value or key that is not finite reaches exactly the rows of its sequence that keep it."""
    gen = torch.Generator().manual_seed(D + G)
    kind = fa.FLEX_MASK_WINDOW_SINKS if window else fa.FLEX_MASK_CAUSAL
    lens = [37, 260, last]  # the longer last one: kernels of many kv tiles
    window += last if window and last > 50 else 0
    qs = running(lens)
    q, k, v = (tokens(gen, qs[-1], h, D, "thd") for h in (2 * G, 2, 2))
    plan = fa.flex_packed_plan_create(ints(qs), None, qs[-1], None, 2 * G, 2, kind, window, sinks)
    clean = fa.flex_attention_packed_fwd(q, k, v, plan)
    pos = torch.arange(260, device="cuda")
    keep = row_keep(pos, torch.tensor([at], device="cuda"), kind, window, sinks)[:, 0]
    hit = torch.zeros(qs[-1], dtype=torch.bool, device="cuda")
    hit[37:297] = keep
    for value in (math.nan, math.inf, -math.inf):
        bad = v.clone()
        bad[0, 1, 37 + at, 7] = value
        out, lse = fa.flex_attention_packed_fwd(q, k, bad, plan)
        assert torch.equal(lse, clean[1])
        assert torch.equal(out[:, :G], clean[0][:, :G])                   # the other key head's
        mine, was = out[0, G:], clean[0][0, G:]
        assert torch.equal(mine[:, ~hit], was[:, ~hit])
        others = [d for d in range(D) if d != 7]
        assert torch.equal(mine[:, hit][..., others], was[:, hit][..., others])
        assert not mine[:, hit, 7].isfinite().any()
        assert mine[:, hit, 7].isnan().all() or not math.isnan(value)
    bad = k.clone()
    bad[0, 1, 37 + at, 3] = math.nan
    out, lse = fa.flex_attention_packed_fwd(q, bad, v, plan)
    assert torch.equal(out[0, G:, ~hit], clean[0][0, G:, ~hit]) and torch.equal(lse[0, G:, ~hit], clean[1][0, G:, ~hit])
    assert out[0, G:, hit].isnan().all() and lse[0, G:, hit].isnan().all()
    # all of the other sequences' keys and values
    kn, vn = k.clone(), v.clone()
    for x in (kn, vn):
        x[:, :, :37] = math.nan
        x[:, :, 297:] = math.inf
    out, lse = fa.flex_attention_packed_fwd(q, kn, vn, plan)
    assert torch.equal(out[:, :, 37:297], clean[0][:, :, 37:297]) and torch.equal(lse[:, :, 37:297], clean[1][:, :, 37:297])


@pytest.mark.parametrize("pad", [8, 16, 24])
def test_strides(pad):
    """Tensors within larger ones, with strides that are multiples of 16 but not 32 bytes; the result in place."""
    gen = torch.Generator().manual_seed(pad)
    qs = running([100, 57])
    wide = [torch.randn((1, 157, h, 64 + pad), generator=gen).to(BF16).cuda() for h in (6, 2, 2)]
    q, k, v = (x[..., :64].transpose(1, 2) for x in wide)
    big = torch.full((1, 6, 157, 64 + pad), 77.0, dtype=BF16, device="cuda")
    compare(q, k, v, qs, qs, out=big[..., :64])
    assert (big[..., 64:] == 77).all()


def test_starts_that_do_not_ascend():
    """No access outside of the tensors, whatever the starts say; sequences in order are computed all the same."""
    gen = torch.Generator().manual_seed(4)
    q, k, v = tokens(gen, 60, 4, 64, "thd"), tokens(gen, 60, 2, 64, "thd"), tokens(gen, 60, 2, 64, "thd")
    for qs, ks in (([0, 50, 10, 60], [0, 50, 10, 60]), ([-5, 20, 900, 60], [0, 20, 40, 60]), ([0, 20, 40, 60], [7, -3, 900, 60]),
                   ([60, 0, 60, 0, 60, 0, 60], [0, 60, 0, 60, 0, 60, 0])):
        plan = fa.flex_packed_plan_create(ints(qs), ints(ks), 60, 60, 4, 2)
        fa.flex_attention_packed_fwd(q, k, v, plan)
    assert fa.flex_device_status() == fa.FLEX_OK


def test_streams_graphs_and_repeats():
    """One plan on several streams at once and in graphs; other lengths behind the same graph; equal bits each time."""
    gen = torch.Generator().manual_seed(5)
    lens = [[500, 20, 300, 180], [10, 600, 0, 390]]
    T, Hq, Hk, D = 1000, 8, 2, 128
    q, k, v = (tokens(gen, T, h, D, "thd") for h in (Hq, Hk, Hk))
    plans = [fa.flex_packed_plan_create(starts_of(n), None, T, None, Hq, Hk) for n in lens]
    want = [fa.flex_attention_packed_fwd(q, k, v, p) for p in plans]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [fa.flex_attention_packed_fwd(q, k, v, plans[0]), fa.flex_attention_packed_fwd(q, k, v, plans[1], stream=streams[0]),
               fa.flex_attention_packed_fwd(q, k, v, plans[0], stream=streams[1].cuda_stream)]
        torch.cuda.synchronize()
        for (o, l_), (wo, wl) in zip(got, (want[0], want[1], want[0])):
            assert torch.equal(o, wo) and torch.equal(l_, wl)
    starts = starts_of(lens[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = fa.flex_packed_plan_create(starts, None, T, None, Hq, Hk)
        out, lse = fa.flex_attention_packed_fwd(q, k, v, plan)
    for i in (1, 0, 1):
        starts.copy_(starts_of(lens[i]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


FIRST_CALL = """
import torch
from block_sparse_masked_blockmask_gb300 import flexattn as fa
starts = torch.tensor([0, 70, 70, 150], dtype=torch.int32, device="cuda")
zero = torch.zeros(3, dtype=torch.int32, device="cuda")
table = torch.arange(30, dtype=torch.int32, device="cuda").view(3, 10)
q, k, v = (torch.randn((1, 150, h, 64), device="cuda").bfloat16().transpose(1, 2) for h in (6, 2, 2))
c = fa.flex_kv_cache_create(30, 2, 64, 16, torch.uint8)

def step():
    fa.flex_kv_cache_append_packed(c, k, v, starts, table, zero)
    k2, v2 = fa.flex_kv_cache_read(c, table, starts, 150)
    plan = fa.flex_packed_plan_create(starts, None, 150, None, 6, 2)
    return fa.flex_attention_packed_fwd(q, k2, v2, plan)

g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
want = step()
assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and want[0].isfinite().all()
assert fa.flex_device_status() == fa.FLEX_OK
print("captured")
"""


def test_first_calls_of_a_process_are_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_tokens_past_32_bits():
    """Heads whose strides pass 2^31 elements: as the same values close together."""
    gen = torch.Generator().manual_seed(6)
    wide = torch.empty(3 * 2**30, dtype=BF16, device="cuda")
    qs = running([150, 20])
    far = [wide.as_strided((1, h, 170, 64), (2**31, s, 64, 1), at) for h, s, at in
           ((4, 2**29 + 64, 0), (2, 2**31 + 2**27, 2**16), (2, 2**31 + 2**28, 2**17))]
    near = [tokens(gen, 170, h, 64, "htd") for h in (4, 2, 2)]
    for f, n in zip(far, near):
        f.copy_(n)
    plan = fa.flex_packed_plan_create(ints(qs), None, 170, None, 4, 2)
    out = wide.as_strided((1, 4, 170, 64), (2**31, 2**29 + 128, 64, 1), 2**20)
    a = fa.flex_attention_packed_fwd(*far, plan, out=out)
    b = fa.flex_attention_packed_fwd(*near, plan)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kind", [torch.uint8, torch.float8_e4m3fn, BF16], ids=["int4", "e4m3", "bf16"])
def test_prompt_in_parts_through_a_cache(kind):
    """Prompts in two parts: rotation, append, read back and attention each time, then a decoding step; the second part's
    attention against the formula over what the cache holds."""
    gen = torch.Generator().manual_seed(7)
    H, G, D, page, parts = 2, 3, 64, 16, ([40, 0, 130, 7], [90, 33, 1, 0])
    table, pages = table_of(gen, [9] * 4, 9)
    cache = fa.flex_kv_cache_create(pages, H, D, page, kind)
    inv = fa.flex_rope_frequencies(D)
    past = [0] * 4
    for new in parts:
        at, total = running(new), sum(new)
        q, k, v = (tokens(gen, total, h, D, "thd") for h in (H * G, H, H))
        positions = torch.cat([torch.arange(p, p + n) for p, n in zip(past, new)]).int().cuda()[None]
        q, _ = fa.flex_rope_fwd(q, None, inv, positions)
        fa.flex_kv_cache_append_packed(cache, k, v, ints(at), table, ints(past), inv)
        past = [p + n for p, n in zip(past, new)]
        ks = running(past)
        kc, vc = fa.flex_kv_cache_read(cache, table, ints(ks), ks[-1])
        out, lse = compare(q, kc, vc, at, ks)
    q = tokens(gen, 4, H * G, D, "thd")[0].transpose(0, 1)[:, :, None]           # one row a sequence: [4, Hq, 1, D]
    a, la = fa.flex_kv_cache_attention(q, cache, table, ints(past))
    ro, rl, bo, bl = reference(q[:, :, 0].transpose(0, 1)[None], kc, vc, [0, 1, 2, 3, 4], ks, fa.FLEX_MASK_CAUSAL, 0, 0,
                               fa.FLEX_SCORE_IDENTITY, 0, D**-0.5)
    # the values as read were rounded to bf16 once more, 2^-8 of each
    kd = 2.0**-8 * (q[:, :, 0].transpose(0, 1).double().abs().sum(-1) * kc.abs().amax().double() * D**-0.5)
    assert ((a[:, :, 0].transpose(0, 1).double() - ro).abs() <= bo + (2 * kd[..., None] + 2.0**-8) * vc.abs().amax()).all()
    assert ((la[:, :, 0].t().double() - rl).abs() <= bl + kd).all()
