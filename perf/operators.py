"""Timed cases of the operators around the attention: rotary positions, the
paged key/value cache (append and attention) and attention with a sliding
window and sinks.

Each case names its operator in "op":
  rope     q and k of a batch rotated by their positions, or the gradient of that
  append   new keys (rotated on the way) and values written to a paged cache
  cache    the newest tokens' queries against a paged cache
  sinks    attention over whole sequences with a sliding window and first
           tokens that stay visible, forward or forward and backward
The plain forms below compute the same from elementary torch operations.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of 16 sequences: latency only
        dict(name="rope_step", op="rope", B=16, Hq=32, Hk=8, S=1, D=128, rotary=128, layout="half", dtype="bf16",
             order="bhsd", far=131072, factor=1.0, backward=False),
        # q and k of the largest prompt configuration, projected as [B, S, H, D]
        dict(name="rope_prompt", op="rope", B=2, Hq=32, Hk=32, S=16384, D=128, rotary=128, layout="interleaved",
             dtype="bf16", order="bshd", far=0, factor=1.0, backward=False),
        # gradient of a part of the head, frequencies stretched for long contexts, float32
        dict(name="rope_gradient", op="rope", B=1, Hq=16, Hk=4, S=4099, D=64, rotary=32, layout="half", dtype="fp32",
             order="bhsd", far=0, factor=8.0, backward=True),
        # one new token of 32 sequences, pages half full
        dict(name="append_step", op="append", B=32, H=8, S=1, D=128, page=64, cache="e4m3", dtype="bf16", rotary=128,
             layout="half", past=2047, ragged=False),
        # prompts of four sequences, padded to the longest
        dict(name="append_prompt", op="append", B=4, H=8, S=4095, D=128, page=64, cache="e4m3", dtype="bf16",
             rotary=128, layout="half", past=100, ragged=True),
        # a cache that keeps bf16, small pages, float32 projections, half of the head rotated
        dict(name="append_bf16_cache", op="append", B=3, H=16, S=517, D=64, page=16, cache="bf16", dtype="fp32",
             rotary=32, layout="interleaved", past=33, ragged=True),
        # one sequence's step early on: latency only
        dict(name="cache_step_short", op="cache", B=1, H=8, G=4, Q=1, D=128, length=513, ragged=False, page=64,
             cache="e4m3", window=0, sinks=0, score="identity"),
        # a serving batch, sequences of all lengths, one slot empty
        dict(name="cache_step_batch", op="cache", B=64, H=8, G=4, Q=1, D=128, length=8192, ragged=True, page=64,
             cache="e4m3", window=0, sinks=0, score="identity"),
        # two very long sequences
        dict(name="cache_step_long", op="cache", B=2, H=8, G=8, Q=1, D=128, length=131071, ragged=False, page=128,
             cache="e4m3", window=0, sinks=0, score="identity"),
        # four tokens checked at once, window and sinks, a bf16 cache with small pages, one key head per query head
        dict(name="cache_window_tokens", op="cache", B=16, H=16, G=1, Q=4, D=64, length=8191, ragged=True, page=16,
             cache="bf16", window=1024, sinks=4, score="alibi"),
        # the sliding-window configuration with sinks, forward
        dict(name="sinks_forward", op="sinks", B=2, H=8, S=2048, D=64, dtype="bf16", window=256, sinks=4,
             score="identity", backward=False),
        # a training step's attention on long sequences: forward and gradients
        dict(name="sinks_train", op="sinks", B=1, H=16, S=8192, D=128, dtype="bf16", window=1024, sinks=16,
             score="identity", backward=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("rope", "append", "cache", "cache", "sinks"))
    D = rng.choice((64, 128))
    rotary = rng.choice((D, D, D // 2, D // 4))
    layout = rng.choice(("half", "interleaved"))
    if op == "rope":
        Hk = _log(rng, 1, 32)
        Hq = min(32, Hk * rng.choice((1, 2, 4)))
        S = _log(rng, 1, 16384)
        B = _log(rng, 1, max(1, min(64, 32768 // S)))
        return dict(op=op, B=B, Hq=Hq, Hk=Hk, S=S, D=D, rotary=rotary, layout=layout,
                    dtype=rng.choice(("bf16", "bf16", "fp32")) if B * S <= 16384 else "bf16",
                    order=rng.choice(("bhsd", "bshd")), far=rng.choice((0, 4096, 1 << 20)),
                    factor=rng.choice((1.0, 4.0, 16.0)), backward=rng.random() < 0.4)
    if op == "append":
        S = 1 if rng.random() < 0.3 else _log(rng, 1, 4095)
        B = _log(rng, 1, max(1, min(64, 16380 // S)))
        return dict(op=op, B=B, H=_log(rng, 1, 8), S=S, D=D, page=rng.choice((16, 32, 64, 128, 256)),
                    cache=rng.choice(("e4m3", "e4m3", "bf16")), dtype=rng.choice(("bf16", "bf16", "fp32")),
                    rotary=rng.choice((0, rotary)), layout=layout, past=_log(rng, 1, 2047), ragged=rng.random() < 0.5)
    if op == "cache":
        H = rng.choice((1, 2, 4, 8, 16))
        length = _log(rng, 1, 131071)
        B = _log(rng, 1, max(1, min(64, 4194304 // (H * length))))
        windowed = rng.random() < 0.4
        return dict(op=op, B=B, H=H, G=rng.choice((1, 2, 4, 5, 8, 16)), Q=1 if rng.random() < 0.6 else _log(rng, 2, 8),
                    D=D, length=length, ragged=rng.random() < 0.6, page=rng.choice((16, 32, 64, 128, 256)),
                    cache=rng.choice(("e4m3", "e4m3", "bf16")), window=_log(rng, 1, 4096) if windowed else 0,
                    sinks=rng.choice((0, 1, 4, 17, 128)) if windowed else 0,
                    score=rng.choice(("identity", "softcap", "alibi")))
    S = _log(rng, 1, 8192)
    H = _log(rng, 1, 16)
    B = _log(rng, 1, max(1, min(4, 8192 * 16 // (S * H))))
    return dict(op=op, B=B, H=H, S=S, D=D, dtype=rng.choice(("bf16", "bf16", "fp32")) if S <= 2048 else "bf16",
                window=_log(rng, 16, 1024), sinks=rng.choice((0, 1, 4, 16, 100, 128)), score="identity",
                backward=rng.random() < 0.5)


# -------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _inv_freq(rotary, factor):
    """Radians per position of every pair, base 10000; stretched by parts for factor > 1."""
    f = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)
    if factor == 1.0:
        return f
    turns = 4096 * f / (2 * math.pi)  # within the 4096 positions trained on
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return f * (keep + (1.0 - keep) / factor)


def _attention_scale(factor):
    return 1.0 if factor == 1.0 else 0.1 * math.log(factor) + 1.0


def _lengths(case, most, least=1):
    """Lengths of a ragged batch, from the case alone: the longest first, one empty from eight sequences on."""
    if not case["ragged"]:
        return [most] * case["B"]
    r = random.Random(case["B"] * 1000003 + most)
    n = [most] + [r.randint(min(least, most), most) for _ in range(case["B"] - 1)]
    if case["B"] >= 8:
        n[-1] = 0
    return n


def _past(case):
    r = random.Random(case["B"] * 1000003 + case["past"])
    return [r.randint(0, case["past"]) for _ in range(case["B"])]


def _page_table(gen, pages_of, width):
    """Pages in random order, -1 behind a sequence's last; and how many pages there are."""
    total = sum(pages_of)
    order = torch.randperm(max(1, total), generator=gen, device="cuda").to(torch.int32)
    n = torch.tensor(pages_of, device="cuda")
    at = (n.cumsum(0) - n)[:, None] + torch.arange(width, device="cuda")
    table = torch.where(torch.arange(width, device="cuda") < n[:, None], order[at.clamp(max=max(1, total) - 1)], -1)
    return table.to(torch.int32).contiguous(), max(1, total)


def _power_scale(amax):
    """The smallest power of two s with amax / s <= 448 = 1.75 * 2^8 (2^-126 at least)."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    return torch.ldexp(torch.ones_like(amax), e)


def _pool(gen, pages, case):
    """Cache contents as a program has them: codes and scales of normal values whose size varies from page to page."""
    shape = (pages, case["H"], case["page"], case["D"])
    size = torch.exp(0.5 * torch.randn((pages, case["H"], 1, 1), generator=gen, device="cuda"))
    x = torch.randn(shape, generator=gen, device="cuda") * size
    if case["cache"] == "bf16":
        return x.to(torch.bfloat16), None
    scale = _power_scale(x.abs().amax((2, 3)))
    return (x / scale[:, :, None, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = _generator(seed)
    op = case["op"]
    if op == "rope":
        B, S, D, dt = case["B"], case["S"], case["D"], DTYPES[case["dtype"]]
        if case["order"] == "bshd":
            q, k = (_normal(gen, (B, S, h, D), dt).transpose(1, 2) for h in (case["Hq"], case["Hk"]))
        else:
            q, k = (_normal(gen, (B, h, S, D), dt) for h in (case["Hq"], case["Hk"]))
        first = torch.randint(0, case["far"], (B, 1), generator=gen, device="cuda") if case["far"] else \
            torch.zeros((B, 1), device="cuda", dtype=torch.int64)
        positions = (first + torch.arange(S, device="cuda")).to(torch.int32)
        return dict(case=case, q=q, k=k, positions=positions, inv_freq=_inv_freq(case["rotary"], case["factor"]))
    if op == "append":
        B, S, page = case["B"], case["S"], case["page"]
        dt = DTYPES[case["dtype"]]
        past, new = _past(case), _lengths(case, S)
        width = -(-(case["past"] + S) // page)
        table, pages = _page_table(gen, [-(-(p + n) // page) for p, n in zip(past, new)], width)
        k, v = (_normal(gen, (B, S, case["H"], case["D"]), dt).transpose(1, 2) for _ in range(2))
        kp, ks = _pool(gen, pages, case)
        vp, vs = _pool(gen, pages, case)
        s = dict(case=case, k=k, v=v, k_pool=kp, v_pool=vp, k_scale=ks, v_scale=vs, table=table,
                 past=torch.tensor(past, dtype=torch.int32, device="cuda"),
                 new=torch.tensor(new, dtype=torch.int32, device="cuda"),
                 inv_freq=_inv_freq(case["rotary"], 1.0) if case["rotary"] else None)
        return _handles(s)
    if op == "cache":
        B, page = case["B"], case["page"]
        lens = _lengths(case, case["length"])
        table, pages = _page_table(gen, [-(-n // page) for n in lens], -(-case["length"] // page))
        q = _normal(gen, (B, case["H"] * case["G"], case["Q"], case["D"]), torch.bfloat16)
        kp, ks = _pool(gen, pages, case)
        vp, vs = _pool(gen, pages, case)
        s = dict(case=case, q=q, k_pool=kp, v_pool=vp, k_scale=ks, v_scale=vs, table=table,
                 lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        return _handles(s)
    shape = (case["B"], case["H"], case["S"], case["D"])
    q, k, v, g = (_normal(gen, shape, DTYPES[case["dtype"]]) for _ in range(4))
    return _handles(dict(case=case, q=q, k=k, v=v, dout=g))


def _handles(s):
    """What a program keeps between calls: the cache object, or the BlockMask of its sizes."""
    if own:
        from block_sparse_masked_blockmask_gb300 import flexattn as fa
        c = s["case"]
        if "k_pool" in s:
            s["kv"] = fa.KVCache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
        else:
            s["mask"] = fa.flex_block_mask_create(fa.FLEX_MASK_WINDOW_SINKS, c["B"], c["H"], c["S"], c["S"],
                                                  window=c["window"], sinks=c["sinks"])
            s["mask_q"] = fa.flex_block_mask_transpose(s["mask"]) if c["backward"] else None
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return {"rope": _rope, "append": _append, "cache": _cache, "sinks": _sinks}[state["case"]["op"]](state)


def _run_own(s):
    from block_sparse_masked_blockmask_gb300 import flexattn as fa
    c = s["case"]
    if c["op"] == "rope":
        f = fa.flex_rope_bwd if c["backward"] else fa.flex_rope_fwd
        return f(s["q"], s["k"], s["inv_freq"], s["positions"],
                 layout=fa.FLEX_ROPE_HALF if c["layout"] == "half" else fa.FLEX_ROPE_INTERLEAVED,
                 attention_scale=_attention_scale(c["factor"]))
    if c["op"] == "append":
        fa.flex_kv_cache_append(s["kv"], s["k"], s["v"], s["table"], s["past"], s["new"], inv_freq=s["inv_freq"],
                                layout=fa.FLEX_ROPE_HALF if c["layout"] == "half" else fa.FLEX_ROPE_INTERLEAVED)
        return s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"]
    if c["op"] == "cache":
        kind = fa.FLEX_MASK_WINDOW_SINKS if c["window"] else fa.FLEX_MASK_CAUSAL
        score = {"identity": fa.FLEX_SCORE_IDENTITY, "softcap": fa.FLEX_SCORE_SOFTCAP,
                 "alibi": fa.FLEX_SCORE_ALIBI}[c["score"]]
        return fa.flex_kv_cache_attention(s["q"], s["kv"], s["table"], s["lens"], mask_kind=kind, window=c["window"],
                                          sinks=c["sinks"], score_kind=score, score_param=30.0)
    out, lse = fa.flex_attention_fwd(s["q"], s["k"], s["v"], s["mask"])
    if not c["backward"]:
        return out, lse
    return (out, lse) + tuple(fa.flex_attention_bwd(s["q"], s["k"], s["v"], out, lse, s["dout"], s["mask"],
                                                    s["mask_q"]))


def _rotate(x, positions, inv_freq, layout, scale, inverse=False):
    """x [B, H, S, D] in 32 bits, rotated; the angles in 64."""
    angle = positions[:, None, :, None].double() * inv_freq
    cos, sin = (angle.cos() * scale).float(), (angle.sin() * (-scale if inverse else scale)).float()
    r = 2 * inv_freq.numel()
    part, rest = x[..., :r].float(), x[..., r:].float()
    if layout == "half":
        a, b = part[..., :r // 2], part[..., r // 2:]
        part = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((part, rest), -1)


def _rope(s):
    c = s["case"]
    args = (s["positions"], s["inv_freq"], c["layout"], _attention_scale(c["factor"]), c["backward"])
    return _rotate(s["q"], *args).to(s["q"].dtype), _rotate(s["k"], *args).to(s["k"].dtype)


def _append(s):
    c = s["case"]
    S, page = c["S"], c["page"]
    t = torch.arange(S, device="cuda")
    positions = s["past"][:, None] + t
    valid = t < s["new"][:, None]
    k, v = s["k"].float(), s["v"].float()
    if s["inv_freq"] is not None:
        k = _rotate(s["k"], positions, s["inv_freq"], c["layout"], 1.0)
    return _write(s["k_pool"], s["k_scale"], k, s, positions, valid, page), \
        _write(s["v_pool"], s["v_scale"], v, s, positions, valid, page), s["k_scale"], s["v_scale"]


def _write(pool, scale, x, s, positions, valid, page):
    slot, at = (positions // page).long(), (positions % page).long()
    ids = s["table"].gather(1, slot.clamp(max=s["table"].shape[1] - 1)).long()
    b, t = valid.nonzero(as_tuple=True)
    tokens = x[b, :, t]                                                   # [tokens, H, D]
    if scale is not None:
        amax = torch.zeros((pool.shape[0], pool.shape[1]), device="cuda")
        amax.index_reduce_(0, ids[b, t], tokens.abs().amax(-1), "amax")
        # the one page of a sequence that already holds tokens: its scale only grows
        held = (s["past"] % page > 0) & (s["new"] > 0)
        seq = held.nonzero()[:, 0]
        old = s["table"][seq, (s["past"][seq] // page).long()].long()
        grown = _power_scale(amax)
        before = scale[old]
        after = torch.maximum(before, grown[old])
        filled = torch.arange(page, device="cuda") < (s["past"][seq] % page)[:, None]
        codes = pool[old].float()
        again = (codes * (before / after)[:, :, None, None]).to(pool.dtype).float()
        pool[old] = torch.where(filled[:, None, :, None], again, codes).to(pool.dtype)
        touched = torch.zeros(pool.shape[0], dtype=torch.bool, device="cuda")
        touched[ids[b, t]] = True
        scale.copy_(torch.where(touched[:, None], grown, scale))
        scale[old] = after
        tokens = tokens / scale[ids[b, t]][:, :, None]
    pool[ids[b, t], :, at[b, t]] = tokens.to(pool.dtype)
    return pool


def _gathered(pool, scale, table):
    """The cache of every sequence as [B, H, positions, D] in 32 bits."""
    ids = table.clamp(min=0).long()
    x = pool[ids].float()
    if scale is not None:
        x = x * scale[ids][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _slopes(heads, dtype=torch.float32):
    return 2.0 ** (-8.0 * torch.arange(1, heads + 1, device="cuda", dtype=dtype) / heads)


def _cache(s):
    c = s["case"]
    B, H, G, Q, D = c["B"], c["H"], c["G"], c["Q"], c["D"]
    k, v = _gathered(s["k_pool"], s["k_scale"], s["table"]), _gathered(s["v_pool"], s["v_scale"], s["table"])
    q = s["q"].float().reshape(B, H, G * Q, D)
    x = (q @ k.transpose(2, 3)).reshape(B, H, G, Q, -1) / math.sqrt(D)
    kv = torch.arange(k.shape[2], device="cuda")
    pos = (s["lens"][:, None] - Q + torch.arange(Q, device="cuda"))[:, None, None, :, None]
    if c["score"] == "softcap":
        x = 30.0 * torch.tanh(x / 30.0)
    elif c["score"] == "alibi":
        x = x - _slopes(H * G).reshape(1, H, G, 1, 1) * (pos - kv).float()
    keep = kv <= pos
    if c["window"]:
        keep = keep & ((pos - kv < c["window"]) | (kv < c["sinks"]))
    x = x.masked_fill(~keep, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    seen = kv < s["lens"][:, None]                                      # what lies behind the last token is not read
    v = v.masked_fill(~seen[:, None, :, None], 0.0)
    out = (p.reshape(B, H, G * Q, -1) @ v).reshape(B, H, G, Q, D)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + total.log())[..., 0]
    return out.reshape(B, H * G, Q, D).to(s["q"].dtype), lse.reshape(B, H * G, Q)


def _sinks(s):
    c = s["case"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    i = torch.arange(c["S"], device="cuda")
    far = i[:, None] - i
    keep = (far >= 0) & ((far < c["window"]) | (i < c["sinks"]))
    scale = 1.0 / math.sqrt(c["D"])
    x = ((q @ k.transpose(2, 3)) * scale).masked_fill(~keep, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0]
    p = p / total
    out = p @ v
    dt = s["q"].dtype
    if not c["backward"]:
        return out.to(dt), lse
    g = s["dout"].float()
    dv = p.transpose(2, 3) @ g
    ds = p * (g @ v.transpose(2, 3) - (g * out).sum(-1, keepdim=True))
    dq, dk = scale * (ds @ k), scale * (ds.transpose(2, 3) @ q)
    return out.to(dt), lse, dq.to(dt), dk.to(dt), dv.to(dt)


# ----------------------------------------------------------------- the work
def work(case):
    op, D = case["op"], case["D"]
    if op == "rope":
        n = case["B"] * (case["Hq"] + case["Hk"]) * case["S"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2.0 * n * D * size + 4 * case["B"] * case["S"], "flops": 3.0 * n * case["rotary"]}
    if op == "append":
        tokens = sum(_lengths(case, case["S"]))
        size, held = 2 if case["dtype"] == "bf16" else 4, 1 if case["cache"] == "e4m3" else 2
        n = 2.0 * tokens * case["H"] * D
        return {"bytes": n * (size + held) + 8.0 * case["H"] * tokens / case["page"], "flops": n}
    if op == "cache":
        lens = _lengths(case, case["length"])
        Q, W = case["Q"], case["window"]
        rows, seen = 0, 0  # (row, key) pairs, and keys that some row sees
        for n in lens:
            for t in range(Q):
                p = n - Q + t
                if p >= 0:
                    rows += p + 1 if not W else min(p + 1, W + min(case["sinks"], max(0, p + 1 - W)))
            seen += n if not W else min(n, W + Q - 1 + min(case["sinks"], max(0, n - W - Q + 1)))
        held = 1 if case["cache"] == "e4m3" else 2
        heads = case["H"] * case["G"]
        return {"bytes": 2.0 * seen * case["H"] * D * held + case["B"] * Q * heads * (4.0 * D + 4),
                "flops": 4.0 * rows * heads * D}
    S, W = case["S"], case["window"]
    pairs = sum(min(p + 1, W + min(case["sinks"], max(0, p + 1 - W))) for p in range(S)) * case["B"] * case["H"]
    n = case["B"] * case["H"] * S * D * (2.0 if case["dtype"] == "bf16" else 4.0)
    back = case["backward"]
    return {"bytes": n * (8 if back else 4), "flops": pairs * D * (14.0 if back else 4.0)}


# ---------------------------------------------------------- in 64 bits, apart
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "cache": _exact_cache, "sinks": _exact_sinks}[case["op"]](s)


def _turned(x, positions, inv_freq, layout, scale):
    """Complex form: (x0 + i x1) scale exp(i position freq)."""
    r = 2 * inv_freq.numel()
    y = x.double().clone()
    first, second = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    angle = positions.double()[:, None, :, None] * inv_freq
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.full_like(angle, scale), angle)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rope(s):
    c = s["case"]
    sign = -1.0 if c["backward"] else 1.0
    return tuple(_turned(x, s["positions"], sign * s["inv_freq"], c["layout"], _attention_scale(c["factor"]))
                 for x in (s["q"], s["k"]))


def _nearest_code(x):
    """Nearest value of a float with 3 fraction bits and exponents from -6, ties to even."""
    e = torch.frexp(x.abs())[1].double() - 1
    step = 2.0 ** (e.clamp(min=-6.0) - 3.0)
    return torch.round(x / step) * step


def _exact_append(s):
    c = s["case"]
    page = c["page"]
    results = []
    for x, pool, scale, rotated in ((s["k"], s["k_pool"], s["k_scale"], s["inv_freq"] is not None),
                                    (s["v"], s["v_pool"], s["v_scale"], False)):
        held = pool.double()
        sc = None if scale is None else scale.double()
        if rotated:
            pos = s["past"][:, None] + torch.arange(c["S"], device="cuda")
            x = _turned(x, pos, s["inv_freq"], c["layout"], 1.0)
        x = x.double()
        for b, (p, n) in enumerate(zip(_past(c), _lengths(c, c["S"]))):
            done = 0
            while done < n:
                first = p + done
                take = min(n - done, page - first % page)
                pid = int(s["table"][b, first // page])
                at = first % page
                new = x[b, :, done:done + take]
                if sc is not None:
                    amax = new.abs().amax((1, 2))
                    want = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)))
                    want = torch.where(amax / want > E4M3_MAX, 2 * want, want)
                    want = torch.where(amax / (0.5 * want) <= E4M3_MAX, 0.5 * want, want)
                    if at:
                        want = torch.maximum(want, sc[pid])
                        held[pid, :, :at] = _nearest_code(held[pid, :, :at] * (sc[pid] / want)[:, None, None])
                    sc[pid] = want
                    new = _nearest_code(new / want[:, None, None])
                held[pid, :, at:at + take] = new
                done += take
        results.append((held, sc))
    (k, ks), (v, vs) = results
    return k, v, ks, vs


def _exact_cache(s):
    c = s["case"]
    H, G, Q, D = c["H"], c["G"], c["Q"], c["D"]
    outs, lses = [], []
    for b, n in enumerate(_lengths(c, c["length"])):
        out = torch.zeros((H * G, Q, D), dtype=torch.float64, device="cuda")
        lse = torch.full((H * G, Q), -math.inf, dtype=torch.float64, device="cuda")
        if n:
            ids = s["table"][b, :-(-n // c["page"])].long()
            k, v = (p[ids].double() if sc is None else p[ids].double() * sc[ids].double()[:, :, None, None]
                    for p, sc in ((s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"])))
            k, v = (x.permute(1, 0, 2, 3).reshape(H, -1, D)[:, :n] for x in (k, v))
            at = torch.arange(n, device="cuda")
            for t in range(Q):
                pos = n - Q + t
                if pos < 0:
                    continue
                seen = at <= pos
                if c["window"]:
                    seen &= (at > pos - c["window"]) | (at < c["sinks"])
                idx = seen.nonzero()[:, 0]
                qt = s["q"][b, :, t].double().reshape(H, G, D)
                x = torch.einsum("hgd,hnd->hgn", qt, k[:, idx]) * D ** -0.5
                if c["score"] == "softcap":
                    x = 30.0 * torch.tanh(x / 30.0)
                elif c["score"] == "alibi":
                    x = x - _slopes(H * G, torch.float64).reshape(H, G, 1) * (pos - idx).double()
                lse[:, t] = torch.logsumexp(x, -1).reshape(-1)
                out[:, t] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), v[:, idx]).reshape(-1, D)
        outs.append(out)
        lses.append(lse)
    return torch.stack(outs), torch.stack(lses)


def _exact_sinks(s):
    c = s["case"]
    S, D, W = c["S"], c["D"], c["window"]
    q, k, v, g = (s[n].double() for n in ("q", "k", "v", "dout"))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.zeros_like(q), torch.zeros_like(q)
    for a in range(0, S, 256):
        e = min(a + 256, S)
        rows = torch.arange(a, e, device="cuda")[:, None]
        low = max(0, a - W + 1)
        cols = torch.cat((torch.arange(0, min(c["sinks"], low), device="cuda"), torch.arange(low, e, device="cuda")))
        hidden = (cols > rows) | ((rows - cols >= W) & (cols >= c["sinks"]))
        kc, vc = k[:, :, cols], v[:, :, cols]
        x = torch.einsum("bhqd,bhkd->bhqk", q[:, :, a:e], kc) * D ** -0.5
        x[:, :, hidden] = -math.inf
        lse[:, :, a:e] = torch.logsumexp(x, -1)
        p = torch.softmax(x, -1)
        out[:, :, a:e] = torch.einsum("bhqk,bhkd->bhqd", p, vc)
        if c["backward"]:
            ga = g[:, :, a:e]
            dp = torch.einsum("bhqd,bhkd->bhqk", ga, vc)
            ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * D ** -0.5
            dq[:, :, a:e] = torch.einsum("bhqk,bhkd->bhqd", ds, kc)
            dk.index_add_(2, cols, torch.einsum("bhqk,bhqd->bhkd", ds, q[:, :, a:e]))
            dv.index_add_(2, cols, torch.einsum("bhqk,bhqd->bhkd", p, ga))
    return (out, lse, dq, dk, dv) if c["backward"] else (out, lse)
