"""Rotary positions against the complex form in float64, at the tensors'
strides and types, and as the gradient of itself.

Bounds.  The angle is exact to 2^-33 of a turn; rounding it to float32 half
turns adds at most 2^-24 pi, and sine and cosine are within 2 units of 2^-24,
so a rotated value is off by at most 2^-21 of |x0| + |x1| (times the attention
scale) in float32, and is then rounded once: 2^-8 of itself in bf16, 2^-24 in
float32.
"""
import math

import pytest
import torch

from block_sparse_masked_blockmask_gb300 import flexattn as fa

pytestmark = pytest.mark.gpu
DT = {"bf16": (torch.bfloat16, 2.0**-8), "fp32": (torch.float32, 2.0**-24)}


def turned(x, positions, inv_freq, layout, scale, sign=1.0):
    """float64 result, and |x0| + |x1| of every value's pair (0 where nothing turns)."""
    r = 2 * inv_freq.numel()
    y, size = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    a, b = (slice(0, r // 2), slice(r // 2, r)) if layout == fa.FLEX_ROPE_HALF else (slice(0, r, 2), slice(1, r, 2))
    angle = sign * positions.double()[:, None, :, None] * inv_freq
    z = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.full_like(angle, scale), angle)
    size[..., a] = size[..., b] = scale * (y[..., a].abs() + y[..., b].abs())
    y[..., a], y[..., b] = z.real, z.imag
    return y, size


def check(got, want, size, r, what):
    diff = (got.double() - want).abs()
    bound = r * want.abs() + 2.0**-21 * size
    assert (diff <= bound).all(), (what, float((diff - bound).max()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", [fa.FLEX_ROPE_HALF, fa.FLEX_ROPE_INTERLEAVED])
@pytest.mark.parametrize("D,rotary", [(64, 64), (64, 16), (128, 128), (128, 48)])
@pytest.mark.parametrize("B,Hq,Hk,S", [(1, 1, 1, 1), (3, 5, 1, 7), (2, 16, 4, 130), (2, 33, 32, 33), (1, 4, 0, 300)])
def test_rope(B, Hq, Hk, S, D, rotary, layout, dtype):
    dt, r = DT[dtype]
    gen = torch.Generator().manual_seed(B * S + D)
    inv = fa.flex_rope_frequencies(rotary)
    far = torch.randint(-5, 2**31 - 1 - S, (B, 1), generator=gen)
    q = torch.randn((B, S, Hq, D), generator=gen).to(dt).cuda().transpose(1, 2)  # strided
    k = torch.randn((B, Hk, S, D), generator=gen).to(dt).cuda() if Hk else None
    for positions in (None, (far + torch.arange(S)).to(torch.int32).cuda()):
        for scale, f, sign in ((1.0, fa.flex_rope_fwd, 1.0), (1.25, fa.flex_rope_bwd, -1.0)):
            at = positions if positions is not None else torch.arange(S, device="cuda").expand(B, S)
            oq, ok = f(q, k, inv, positions, layout=layout, attention_scale=scale)
            check(oq, *turned(q, at, inv, layout, scale, sign), r, "q")
            assert (ok is None) == (k is None)
            if k is not None:
                check(ok, *turned(k, at, inv, layout, scale, sign), r, "k")


def test_in_place_and_strided_output():
    inv = fa.flex_rope_frequencies(64)
    q = torch.randn((2, 9, 4, 128), device="cuda").bfloat16().transpose(1, 2)
    k = torch.randn((2, 2, 9, 128), device="cuda").bfloat16()
    oq, ok = fa.flex_rope_fwd(q, k, inv)
    wide = torch.full((2, 9, 6, 128), 7.0, device="cuda", dtype=torch.bfloat16)
    fa.flex_rope_fwd(q, None, inv, q_out=wide[:, :, 1:5].transpose(1, 2))
    assert torch.equal(wide[:, :, 1:5].transpose(1, 2), oq)
    assert (wide[:, :, 0] == 7).all() and (wide[:, :, 5] == 7).all()
    fa.flex_rope_fwd(q, k, inv, q_out=q, k_out=k)
    assert torch.equal(q, oq) and torch.equal(k, ok)


def test_gradient_against_differences():
    # loss = sum(w y(x)): linear in x, so (loss(x + e) - loss(x - e)) / 2 is the
    # gradient times e up to the rounding of the values
    inv = fa.flex_rope_frequencies(32)
    gen = torch.Generator().manual_seed(3)
    x, w, e = (torch.randn((2, 3, 5, 64), generator=gen).cuda() for _ in range(3))
    args = dict(layout=fa.FLEX_ROPE_INTERLEAVED, attention_scale=1.5)
    up, down = (fa.flex_rope_fwd(x + s * e, None, inv, **args)[0] for s in (1, -1))
    slope = (w.double() * (up.double() - down.double())).sum() / 2
    dx = fa.flex_rope_bwd(w, None, inv, **args)[0]
    size = 3 * (w.abs() * (x.abs() + e.abs())).double().sum() * 2  # |pair| <= sum of both magnitudes, twice
    assert abs(float((dx.double() * e.double()).sum() - slope)) <= 2.0**-21 * float(size)


def test_frequencies():
    i = torch.arange(0, 64, 2, dtype=torch.float64)
    f = 10000.0 ** (-i / 64)
    get = lambda *a, **k: fa.flex_rope_frequencies(*a, device="cpu", **k)  # noqa: E731
    close = lambda a, b: torch.allclose(a, b, rtol=1e-14, atol=0)  # noqa: E731
    assert close(get(64), f)
    assert close(get(64, scaling=fa.FLEX_ROPE_SCALE_LINEAR, factor=4.0), f / 4)
    assert close(get(64, scaling=fa.FLEX_ROPE_SCALE_BASE, factor=4.0), (10000.0 * 4 ** (64 / 62)) ** (-i / 64))
    turns = 4096 * f / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    assert close(get(64, scaling=fa.FLEX_ROPE_SCALE_PARTS, factor=8.0, original_len=4096),
                 f * (keep + (1 - keep) / 8))


def test_other_stream_and_graph():
    inv = fa.flex_rope_frequencies(128)
    q, k = (torch.randn((1, 8, 40, 128), device="cuda").bfloat16() for _ in range(2))
    want = fa.flex_rope_fwd(q, k, inv)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = fa.flex_rope_fwd(q, k, inv, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = fa.flex_rope_fwd(q, k, inv)
    q.mul_(2)
    g.replay()
    assert torch.equal(got[0], fa.flex_rope_fwd(q, k, inv)[0])
