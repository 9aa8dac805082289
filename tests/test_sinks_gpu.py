"""Sliding window + sinks masks: the BlockMask against brute force, and the
forward and backward against the formulas in float64.

Bounds.  Scores are float32 sums of D exact products: each is off by at most
(D + 8) 2^-24 scale sum |q k|, and so is lse, plus 2^-20 for the exponentials
and their sum.  The bf16 path rounds P (half a step: 2^-8 of each weight) and
its outputs (2^-8 of each); dS is rounded once more, and delta comes from the
rounded out.  So with A the same sums over absolute values,
  |d out| <= 2^-8 |out| + (2^-8 + e) A_out,  and likewise for the gradients,
where e covers the relative error of P that the score errors cause.  The
float32 path splits every operand into three bf16 parts: what it leaves out of
each product is at most 2^-22 of it, 2^-18 of A with the sums.
"""
import itertools
import math

import numpy as np
import pytest
import torch

from block_sparse_masked_blockmask_gb300 import flexattn as fa

pytestmark = pytest.mark.gpu


def dense_mask(q_len, kv_len, window, sinks):
    q, kv = torch.arange(q_len)[:, None], torch.arange(kv_len)
    return (q >= kv) & ((q - kv < window) | (kv < sinks))


def brute_blocks(keep, qb, kvb):
    nq, nk = -(-keep.shape[0] // qb), -(-keep.shape[1] // kvb)
    pad = torch.zeros((nq * qb, nk * kvb), dtype=torch.bool)
    pad[:keep.shape[0], :keep.shape[1]] = keep
    t = pad.reshape(nq, qb, nk, kvb)
    full = t.all(3).all(1)
    return t.any(3).any(1) & ~full, full


def ordered(sel):
    """Per row: the selected blocks ascending, then the others."""
    return torch.sort((~sel).to(torch.int8), dim=1, stable=True).indices.to(torch.int32)


@pytest.mark.parametrize("q_len,kv_len", [(1, 1), (127, 127), (129, 129), (1000, 1000), (200, 700), (700, 200)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 3), (1, 0), (1, 1), (100, 4), (128, 128), (64, 200), (257, 129),
                                          (2**31 - 1, 5), (3, 2**31 - 1)])
def test_block_mask(q_len, kv_len, window, sinks):
    keep = dense_mask(q_len, kv_len, window, sinks)
    for qb, kvb in ((128, 128), (16, 64), (256, 32)):
        bm = fa.flex_block_mask_create(fa.FLEX_MASK_WINDOW_SINKS, 1, 2, q_len, kv_len, qb, window=window, sinks=sinks,
                                       kv_block=kvb)
        part, full = brute_blocks(keep, qb, kvb)
        got = bm.as_numpy()
        for h in range(2):
            assert np.array_equal(got["kv_num_blocks"][0, h], part.sum(1).int().numpy())
            assert np.array_equal(got["full_kv_num_blocks"][0, h], full.sum(1).int().numpy())
            assert np.array_equal(got["kv_indices"][0, h], ordered(part).numpy())
            assert np.array_equal(got["full_kv_indices"][0, h], ordered(full).numpy())


def reference(q, k, v, g, keep, score, cap, scale):
    """float64 out, lse, gradients, the same sums over absolute values, and the bound of the scores' errors."""
    q, k, v, g = (x.double() for x in (q, k, v, g))
    H, D = q.shape[1], q.shape[3]
    t = scale * (q @ k.transpose(2, 3))
    size = scale * (q.abs() @ k.abs().transpose(2, 3))
    s, slope = t, torch.ones_like(t)
    if score == fa.FLEX_SCORE_SOFTCAP:
        s = cap * torch.tanh(t / cap)
        slope = 1 - torch.tanh(t / cap) ** 2
    elif score == fa.FLEX_SCORE_ALIBI:
        h = torch.arange(1, H + 1, device=q.device, dtype=torch.float64)
        far = torch.arange(q.shape[2], device=q.device)[:, None] - torch.arange(k.shape[2], device=q.device)
        s = t - (2.0 ** (-8.0 * h / H)).reshape(1, H, 1, 1) * far
        size = size + far.abs()
    s = s.masked_fill(~keep, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(keep, (s - lse[..., None]).exp(), 0.0)
    e_s = ((D + 8) * 2.0**-24 * torch.where(keep, size, 0.0)).amax(-1)
    out = p @ v
    dv = p.transpose(2, 3) @ g
    dp = g @ v.transpose(2, 3)
    delta = (g * out).sum(-1, keepdim=True)
    ds = p * (dp - delta) * slope
    # per pair: |dS| and what the rounding of out does to delta, and P times the size of dP
    ads = p * slope * ((dp - delta).abs() + (g.abs() * out.abs()).sum(-1, keepdim=True))
    adp = p * slope * (g.abs() @ v.abs().transpose(2, 3) + (g * out).abs().sum(-1, keepdim=True))
    absolute = dict(out=p @ v.abs(), dv=p.transpose(2, 3) @ g.abs(), dq=scale * (ads @ k.abs()),
                    dk=scale * (ads.transpose(2, 3) @ q.abs()))
    product = dict(out=absolute["out"], dv=absolute["dv"], dq=scale * (adp @ k.abs()),
                   dk=scale * (adp.transpose(2, 3) @ q.abs()))
    return dict(out=out, lse=lse, dq=scale * (ds @ k), dk=scale * (ds.transpose(2, 3) @ q), dv=dv), absolute, product, e_s


CASES = [(w, s) + x for (w, s), x in zip(
    [(0, 0), (0, 3), (1, 0), (1, 1), (16, 4), (100, 4), (128, 128), (300, 17), (64, 200), (2**31 - 1, 5), (40, 2**31 - 1),
     (256, 4), (257, 130)],
    itertools.cycle([(130, 130), (1, 1), (129, 129), (500, 500), (300, 200), (130, 300), (257, 257)]))]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks,q_len,kv_len", CASES + [(100, 4, 1000, 1000), (256, 4, 700, 700)])
def test_forward_and_backward(window, sinks, q_len, kv_len, D, dtype):
    B, H = 2, 3
    scale = 1.0 / math.sqrt(D)
    gen = torch.Generator().manual_seed(q_len * 7 + D)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v, g = (torch.randn((B, H, n, D), generator=gen).to(dt).cuda() for n in (q_len, kv_len, kv_len, q_len))
    keep = dense_mask(q_len, kv_len, window, sinks).cuda()
    for score in (fa.FLEX_SCORE_IDENTITY, fa.FLEX_SCORE_ALIBI):
        ref, absolute, product, e_s = reference(q, k, v, g, keep, score, 0.0, scale)
        for blocks in ((128, None), (64, 256)):
            bm = fa.flex_block_mask_create(fa.FLEX_MASK_WINDOW_SINKS, B, H, q_len, kv_len, blocks[0], window=window,
                                           sinks=sinks, kv_block=blocks[1])
            out, lse = fa.flex_attention_fwd(q, k, v, bm, score)
            got = dict(zip(("dq", "dk", "dv"), fa.flex_attention_bwd(q, k, v, out, lse, g, bm,
                                                                     fa.flex_block_mask_transpose(bm), score)))
            assert fa.flex_device_status() == fa.FLEX_OK
            got["out"] = out
            empty = ~keep.any(-1)
            assert torch.isneginf(lse[:, :, empty]).all() and (out[:, :, empty] == 0).all()
            assert (got["dq"][:, :, empty] == 0).all()
            live = ~empty
            e_lse = (lse.double() - ref["lse"]).abs()[:, :, live]
            assert (e_lse <= e_s[:, :, live] + 2.0**-20 * (1 + ref["lse"][:, :, live].abs())).all(), \
                (score, blocks, float(e_lse.max()))
            e_p = 2 * float(e_s.max()) + 2.0**-18 if live.any() else 0.0  # relative error of a recomputed P
            for name, x in got.items():
                diff = (x.double() - ref[name]).abs()
                r = 2.0**-8 if dtype == "bf16" else 2.0**-18
                bound = r * ref[name].abs() + 2 * r * absolute[name] + (e_p + 2.0**-18) * product[name]
                assert (diff <= bound + 1e-30).all(), (name, score, blocks, float((diff - bound).max()))


def test_no_sinks_is_the_sliding_window():
    q, k, v = (torch.randn((1, 2, 700, 64), device="cuda").bfloat16() for _ in range(3))
    a = fa.flex_block_mask_create(fa.FLEX_MASK_WINDOW_SINKS, 1, 2, 700, 700, window=100)
    b = fa.flex_block_mask_create(fa.FLEX_MASK_SLIDING_WINDOW, 1, 2, 700, 700, window=100)
    for key, x in a.as_numpy().items():
        assert np.array_equal(x, b.as_numpy()[key])
    (oa, la), (ob, lb) = fa.flex_attention_fwd(q, k, v, a), fa.flex_attention_fwd(q, k, v, b)
    # the older kind sums its weights after rounding them: each off by 2^-8 at most
    assert (oa.float() - ob.float()).abs().max() <= 3 * 2.0**-8 * v.float().abs().max()
    assert (la - lb).abs().max() <= 2.0**-8 * 1.01


def test_host_entry_point_and_options():
    B, H, S, D = 1, 4, 333, 64
    q, k, v = (torch.randn((B, H, S, D)).bfloat16().pin_memory() for _ in range(3))
    out, lse = torch.empty_like(q).pin_memory(), torch.empty((B, H, S)).pin_memory()
    fa.flex_attention_fwd_host(q, k, v, fa.DeviceBuffers(B, H, S, S, D, torch.bfloat16), fa.FLEX_MASK_WINDOW_SINKS, out,
                               lse, window=50, sinks=7, chunks=3)
    torch.cuda.synchronize()
    bm = fa.flex_block_mask_create(fa.FLEX_MASK_WINDOW_SINKS, B, H, S, S, window=50, sinks=7)
    o, l_, m = fa.flex_attention_fwd_opts(q.cuda(), k.cuda(), v.cuda(), bm, output_max=True)
    assert torch.equal(o.cpu(), out) and torch.equal(l_.cpu(), lse)
    x = (q.double() @ k.double().transpose(2, 3)) / math.sqrt(D)
    x = x.masked_fill(~dense_mask(S, S, 50, 7), -math.inf)
    assert (m.cpu().double() - x.amax(-1)).abs().max() <= 1e-4


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("score", [fa.FLEX_SCORE_IDENTITY, fa.FLEX_SCORE_SOFTCAP, fa.FLEX_SCORE_ALIBI])
def test_as_the_older_kinds(score, D, dtype):
    """Every score_mod, without sinks against the sliding window and with a window of all tokens against causal:
    the same products, summed in float32 in another order at most.  The older bf16 forward sums rounded weights
    (2^-8 of lse, and of out beside its own rounding and the weights').  The gradients of equal inputs differ by a
    last rounding and by float32 sums: 2^-12 of the largest covers those of 500 terms."""
    S, dt = 500, torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator().manual_seed(score * 10 + D)
    q, k, v, g = (torch.randn((2, 3, S, D), generator=gen).to(dt).cuda() for _ in range(4))
    r = 2.0**-8 if dtype == "bf16" else 2.0**-16
    for new, old in ((dict(window=150), dict(mask_kind=fa.FLEX_MASK_SLIDING_WINDOW, window=150)),
                     (dict(window=S, sinks=9), dict(mask_kind=fa.FLEX_MASK_CAUSAL))):
        a = fa.flex_block_mask_create(fa.FLEX_MASK_WINDOW_SINKS, 2, 3, S, S, **new)
        b = fa.flex_block_mask_create(B=2, H=3, q_len=S, kv_len=S, **old)
        (oa, la), (ob, lb) = (fa.flex_attention_fwd(q, k, v, m, score, 7.0) for m in (a, b))
        assert (oa.float() - ob.float()).abs().max() <= 4 * r * v.float().abs().max()
        assert ((la - lb).abs() <= 1.01 * r * (1 + lb.abs() * (0 if dtype == "bf16" else 1))).all()
        ga, gb = (fa.flex_attention_bwd(q, k, v, ob, lb, g, m, fa.flex_block_mask_transpose(m), score, 7.0)
                  for m in (a, b))
        for x, y in zip(ga, gb):
            x, y = x.float(), y.float()
            assert ((x - y).abs() <= 2 * r * y.abs() + 2.0**-12 * y.abs().max()).all()


def test_training_step_with_rotary_positions():
    """Rotation, attention, its gradients and the rotation back, in float32, against the formula of all of it in
    float64; the formula against differences.  Beside the attention's own bounds: a rotated value is off by 2^-21
    of its pair, which moves scores by less than the bound of their own rounding and gradients by 2^-20 of the sum
    of their terms' sizes; turning back adds up the bounds of a pair."""
    B, H, S, D, rotary, window, sinks = 2, 3, 300, 64, 32, 70, 5
    scale = 1.0 / math.sqrt(D)
    gen = torch.Generator().manual_seed(5)
    q, k, v, g = (torch.randn((B, H, S, D), generator=gen).cuda() for _ in range(4))
    keep = dense_mask(S, S, window, sinks).cuda()
    inv = fa.flex_rope_frequencies(rotary)
    at = torch.arange(1000, 1000 + S, dtype=torch.int32, device="cuda").expand(B, S).contiguous()
    bm = fa.flex_block_mask_create(fa.FLEX_MASK_WINDOW_SINKS, B, H, S, S, window=window, sinks=sinks)
    qr, kr = fa.flex_rope_fwd(q, k, inv, at)
    out, lse = fa.flex_attention_fwd(qr, kr, v, bm)
    dqr, dkr, dv = fa.flex_attention_bwd(qr, kr, v, out, lse, g, bm, fa.flex_block_mask_transpose(bm))
    dq, dk = fa.flex_rope_bwd(dqr, dkr, inv, at)

    def turn(x, sign):
        y, h = x.double().clone(), rotary // 2
        angle = sign * at.double()[:, None, :, None] * inv
        z = torch.complex(y[..., :h], y[..., h:rotary]) * torch.polar(torch.ones_like(angle), angle)
        y[..., :h], y[..., h:rotary] = z.real, z.imag
        return y

    def pairs(x):
        y, h = x.clone(), rotary // 2
        y[..., :h] = y[..., h:rotary] = x[..., :h] + x[..., h:rotary]
        return y

    ref, absolute, product, e_s = reference(turn(q, 1), turn(k, 1), v, g, keep, fa.FLEX_SCORE_IDENTITY, 0.0, scale)
    e_p = 4 * float(e_s.max()) + 2.0**-18
    bound = {n: 2.0**-18 * (ref[n].abs() + 2 * absolute[n]) + 2.0**-20 * absolute[n] + (e_p + 2.0**-18) * product[n]
             for n in ("out", "dq", "dk", "dv")}
    want = dict(out=ref["out"], dv=ref["dv"], dq=turn(ref["dq"], -1), dk=turn(ref["dk"], -1))
    for n in ("dq", "dk"):
        bound[n] = pairs(bound[n]) + 2.0**-21 * pairs(ref[n].abs())
    for n, x in dict(out=out, dq=dq, dk=dk, dv=dv).items():
        diff = (x.double() - want[n]).abs()
        assert (diff <= bound[n]).all(), (n, float((diff - bound[n]).max()))

    def loss(q, k, v):
        s = (scale * (turn(q, 1) @ turn(k, 1).transpose(2, 3))).masked_fill(~keep, -math.inf)
        return float((torch.softmax(s, -1) @ v.double() * g.double()).sum())

    x = [t.double() for t in (q, k, v)]
    step = [torch.randn(t.shape, generator=gen, dtype=torch.float64).cuda() for t in x]
    eps = 1e-5  # the difference is off by about eps^2 times a third derivative, and 1e-16 / eps of the loss
    up, down = (loss(*(t + s * eps * d for t, d in zip(x, step))) for s in (1, -1))
    slope = sum(float((want[n] * d).sum()) for n, d in zip(("dq", "dk", "dv"), step))
    size = sum(float((want[n] * d).abs().sum()) for n, d in zip(("dq", "dk", "dv"), step))
    assert abs((up - down) / (2 * eps) - slope) <= 1e-6 * size


@pytest.mark.parametrize("D", [64, 128])
def test_long_query_side_in_fp32(D):
    """dk and dv of more than 2048 query tiles, which the CUDA cores compute.  Beside the bounds of the short ones a
    column's float32 sum of n terms of no common sign is off by 2^-24 of its partial sums, 8 sqrt(n) of its terms'
    mean size: 2^-21 sqrt(n) of the sum of their sizes, n times over at most, in the mean over n."""
    q_len, kv_len, window, sinks = 2048 * 128 + 130, 200, 70, 3
    gen = torch.Generator().manual_seed(D)
    q, k, v, g = (torch.randn((1, 1, n, D), generator=gen).cuda() for n in (q_len, kv_len, kv_len, q_len))
    keep = dense_mask(q_len, kv_len, window, sinks).cuda()
    bm = fa.flex_block_mask_create(fa.FLEX_MASK_WINDOW_SINKS, 1, 1, q_len, kv_len, window=window, sinks=sinks)
    out, lse = fa.flex_attention_fwd(q, k, v, bm)
    got = dict(zip(("dq", "dk", "dv"), fa.flex_attention_bwd(q, k, v, out, lse, g, bm, fa.flex_block_mask_transpose(bm))))
    got["out"] = out
    ref, absolute, product, e_s = reference(q, k, v, g, keep, fa.FLEX_SCORE_IDENTITY, 0.0, 1.0 / math.sqrt(D))
    e_p = 2 * float(e_s.max()) + 2.0**-18
    terms = keep.sum(0).double().sqrt()[:, None]
    for name, x in got.items():
        diff = (x.double() - ref[name]).abs()
        bound = 2.0**-18 * (ref[name].abs() + 2 * absolute[name]) + (e_p + 2.0**-18) * product[name]
        if name in ("dk", "dv"):
            bound += 2.0**-21 * terms * absolute[name]
        assert (diff <= bound + 1e-30).all(), (name, float((diff - bound).max()))


def check_gradients(q, k, v, g, keep, got, score, r):
    ref, absolute, product, e_s = reference(q, k, v, g, keep, score, 0.0, 1.0 / math.sqrt(q.shape[3]))
    e_p = 2 * float(e_s.max()) + 2.0**-18
    for name, x in got.items():
        diff = (x.double() - ref[name]).abs()
        bound = r * ref[name].abs() + 2 * r * absolute[name] + (e_p + 2.0**-18) * product[name]
        assert (diff <= bound + 1e-30).all(), (name, float((diff - bound).max()))


@pytest.mark.parametrize("H,q_len,kv_len,D,window,sinks", [(1, 4100, 4100, 64, 256, 4), (2, 5000, 5000, 128, 100, 130),
                                                           (1, 3000, 200, 128, 70, 200), (3, 2048, 2048, 64, 0, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_few_heads_and_many_query_tiles(H, q_len, kv_len, D, window, sinks, dtype):
    """dk and dv of the tiles with sinks are summed over parts of the query axis."""
    gen = torch.Generator().manual_seed(q_len + D)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k, v, g = (torch.randn((1, H, n, D), generator=gen).to(dt).cuda() for n in (q_len, kv_len, kv_len, q_len))
    keep = dense_mask(q_len, kv_len, window, sinks).cuda()
    bm = fa.flex_block_mask_create(fa.FLEX_MASK_WINDOW_SINKS, 1, H, q_len, kv_len, window=window, sinks=sinks)
    bq = fa.flex_block_mask_transpose(bm)
    for score in (fa.FLEX_SCORE_IDENTITY, fa.FLEX_SCORE_ALIBI):
        out, lse = fa.flex_attention_fwd(q, k, v, bm, score)
        got = dict(zip(("dq", "dk", "dv"), fa.flex_attention_bwd(q, k, v, out, lse, g, bm, bq, score)))
        assert fa.flex_device_status() == fa.FLEX_OK
        check_gradients(q, k, v, g, keep, got, score, 2.0**-8 if dtype == "bf16" else 2.0**-18)


@pytest.mark.parametrize("score", [fa.FLEX_SCORE_IDENTITY, fa.FLEX_SCORE_SOFTCAP])
@pytest.mark.parametrize("D", [64, 128])
def test_one_head_as_many(D, score):
    """One head, whose tile of sinks is summed over parts, and the same head thirty-two times, where one CTA walks it:
    equal products, another order of float32 sums and one rounding each; and equal bits in a captured call."""
    S, gen = 4100, torch.Generator().manual_seed(D + score)
    q, k, v, g = (torch.randn((1, 1, S, D), generator=gen).bfloat16().cuda() for _ in range(4))

    def run(H):
        x = [t.expand(1, H, S, D).contiguous() for t in (q, k, v, g)]
        bm = fa.flex_block_mask_create(fa.FLEX_MASK_WINDOW_SINKS, 1, H, S, S, window=256, sinks=7)
        bq = fa.flex_block_mask_transpose(bm)
        out, lse = fa.flex_attention_fwd(*x[:3], bm, score, 9.0)
        f = lambda: fa.flex_attention_bwd(*x[:3], out, lse, x[3], bm, bq, score, 9.0)  # noqa: E731
        return f(), f

    (one, again), (many, _) = run(1), run(32)
    for x, y in zip(one, many):
        x, y = x[0, 0].float(), y[0, 5].float()
        assert ((x - y).abs() <= 2.0**-7 * y.abs() + 2.0**-12 * y.abs().max()).all()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        replayed = again()
    graph.replay()
    graph.replay()
    assert all(torch.equal(x, y) for x, y in zip(one, replayed))
