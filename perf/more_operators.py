"""Timed cases of serving with grouped heads and a cache held in 4 bits: prompts
of different lengths packed one behind the other, the cache as it is written
and read back, and the newest tokens' attention against it.

Each case names what is passed through in "op":
  prompt   causal attention over packed sequences, query heads sharing key heads
  store    new tokens of packed sequences written to a paged 4-bit cache (keys
           rotated on the way), and all tokens of the sequences read back from
           it, as the attention over a prompt's next part takes them
  read     the tokens of sequences read back from a cache
  step     one decoding step: each sequence's new token written to the 4-bit
           cache, then the attention of it against the cache
  cache    the newest tokens' attention against the 4-bit cache
The plain forms below compute the same from elementary torch operations.

The 4-bit cache: a token's key has one scale for each 32 neighbouring values,
its value one for all D; a scale is bfloat16(largest magnitude / 7), a code c = 8 + the
nearest whole number to value / scale (halves away from zero).  A token's codes
lie in 16-bit words of four, the first in the lowest bits; word (D / 32) g + j
holds the values 32 j + 4 g to 32 j + 4 g + 3.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # a burst of short prompts, 64 of them: latency, and rows of a tile that come from several heads
        dict(name="prompt_short", op="prompt", N=64, longest=96, ragged=True, past=0, Hk=8, G=4, D=128, window=0,
             sinks=0, score="identity", order="thd"),
        # a prefill batch: twelve prompts of all lengths
        dict(name="prompt_batch", op="prompt", N=12, longest=4096, ragged=True, past=0, Hk=8, G=4, D=128, window=0,
             sinks=0, score="identity", order="thd"),
        # one long prompt, the length of the largest prompt configuration
        dict(name="prompt_long", op="prompt", N=1, longest=16384, ragged=False, past=0, Hk=8, G=4, D=128, window=0,
             sinks=0, score="identity", order="thd"),
        # the next parts of eight long prompts behind what is cached of them; five heads share one, window and sinks
        dict(name="prompt_next_part", op="prompt", N=8, longest=511, ragged=True, past=4099, Hk=4, G=5, D=64, window=1024,
             sinks=4, score="alibi", order="htd"),
        # the next parts of eight prompts stored, and all of them read back for the attention
        dict(name="store_next_part", op="store", N=8, longest=2047, ragged=True, past=2049, H=8, D=128, page=64,
             dtype="bf16", rotary=128, layout="half", out="bf16"),
        # few tokens, small pages, float32 projections, a quarter of the head rotated
        dict(name="store_small", op="store", N=5, longest=131, ragged=True, past=77, H=3, D=64, page=16,
             dtype="fp32", rotary=16, layout="interleaved", out="fp32"),
        # two very long contexts read back
        dict(name="read_long", op="read", N=2, longest=131071, ragged=False, H=8, D=128, page=128, cache="int4",
             out="bf16"),
        # a batch of contexts that lie in 8 bits
        dict(name="read_eight_bits", op="read", N=24, longest=4095, ragged=True, H=8, D=64, page=32, cache="e4m3",
             out="bf16"),
        # one sequence's decoding step early on: latency only
        dict(name="step_short", op="step", B=1, H=8, G=4, Q=1, D=128, length=513, ragged=False, page=64, window=0, sinks=0,
             score="identity", rotary=128, layout="half"),
        # a serving batch's decoding step, sequences of all lengths, one slot empty
        dict(name="step_batch", op="step", B=64, H=8, G=4, Q=1, D=128, length=8192, ragged=True, page=64, window=0,
             sinks=0, score="identity", rotary=128, layout="half"),
        # two very long sequences
        dict(name="cache_long", op="cache", B=2, H=8, G=8, Q=1, D=128, length=131071, ragged=False, page=128, window=0,
             sinks=0, score="identity"),
        # three tokens checked at once, window and sinks, small pages, five heads share one
        dict(name="cache_window_tokens", op="cache", B=16, H=8, G=5, Q=3, D=64, length=8191, ragged=True, page=16,
             window=2048, sinks=4, score="softcap"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "store", "read", "step", "cache"))
    D = rng.choice((64, 128))
    page = rng.choice((16, 32, 64, 128, 256))
    rotary = rng.choice((0, D, D, D // 2, D // 4))
    layout = rng.choice(("half", "interleaved"))
    windowed = rng.random() < 0.4
    window = _log(rng, 1, 4096) if windowed else 0
    sinks = rng.choice((0, 1, 4, 17, 128)) if windowed else 0
    if op == "prompt":
        Hk = rng.choice((1, 2, 4, 8))
        longest = _log(rng, 1, 8192)
        past = 0 if rng.random() < 0.6 else _log(rng, 1, 4096)
        return dict(op=op, N=_log(rng, 1, max(1, min(64, 8192 // longest))), longest=longest, ragged=rng.random() < 0.7,
                    past=past, Hk=Hk, G=rng.choice([g for g in (1, 2, 4, 5, 8, 16) if Hk * g <= 32]), D=D, window=window,
                    sinks=sinks, score=rng.choice(("identity", "identity", "alibi", "softcap")),
                    order=rng.choice(("thd", "htd")))
    if op == "store":
        longest = 1 if rng.random() < 0.2 else _log(rng, 1, 4095)
        return dict(op=op, N=_log(rng, 1, max(1, min(64, 16380 // longest))), longest=longest, ragged=rng.random() < 0.5,
                    past=_log(rng, 1, 2047), H=_log(rng, 1, 8), D=D, page=page, dtype=rng.choice(("bf16", "bf16", "fp32")),
                    rotary=rotary, layout=layout, out=rng.choice(("bf16", "bf16", "fp32")))
    if op == "read":
        longest = _log(rng, 1, 131071)
        H = _log(rng, 1, 8)
        return dict(op=op, N=_log(rng, 1, max(1, min(64, 1048576 // (H * longest)))), longest=longest,
                    ragged=rng.random() < 0.5, H=H, D=D, page=page, cache=rng.choice(("int4", "int4", "e4m3", "bf16")),
                    out=rng.choice(("bf16", "bf16", "fp32")))
    H = rng.choice((1, 2, 4, 8, 16))
    length = _log(rng, 1, 131071)
    case = dict(op=op, B=_log(rng, 1, max(1, min(64, 2097152 // (H * length)))), H=H, G=rng.choice((1, 2, 4, 5, 8, 16)),
                Q=1 if op == "step" or rng.random() < 0.6 else _log(rng, 2, 8), D=D, length=length,
                ragged=rng.random() < 0.6, page=page, window=window, sinks=sinks,
                score=rng.choice(("identity", "softcap", "alibi")))
    return dict(case, rotary=rotary, layout=layout) if op == "step" else case


# -------------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _inv_freq(rotary):
    """Radians per position of every pair, base 10000."""
    return 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)


def _ragged(n, most, ragged, least=1):
    """Lengths of a batch, from the sizes alone: the longest first, one empty from eight sequences on."""
    if not ragged:
        return [most] * n
    r = random.Random(n * 1000003 + most)
    out = [most] + [r.randint(min(least, most), most) for _ in range(n - 1)]
    if n >= 8:
        out[-1] = 0
    return out


def _past(case):
    """Tokens that each sequence has in the cache beforehand; none for a first prompt."""
    r = random.Random(case["N"] * 1000003 + case["past"])
    return [r.randint(0, case["past"]) for _ in range(case["N"])]


def _starts(lens):
    """Where each sequence begins in the packed tokens, and where the last one ends: int32 [N + 1]."""
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _page_table(gen, pages_of, width):
    """Pages in random order, -1 behind a sequence's last; and how many pages there are."""
    total = sum(pages_of)
    order = torch.randperm(max(1, total), generator=gen, device="cuda").to(torch.int32)
    n = torch.tensor(pages_of, device="cuda")
    at = (n.cumsum(0) - n)[:, None] + torch.arange(width, device="cuda")
    table = torch.where(torch.arange(width, device="cuda") < n[:, None], order[at.clamp(max=max(1, total) - 1)], -1)
    return table.to(torch.int32).contiguous(), max(1, total)


def _packed(codes):
    """Codes 0 .. 15 [..., D] as they lie in the cache: uint8 [..., D / 2]."""
    D = codes.shape[-1]
    w = codes.to(torch.uint8).unflatten(-1, (D // 32, 8, 4)).transpose(-3, -2)
    return (w[..., 0::2] | (w[..., 1::2] << 4)).flatten(-3).contiguous()


def _unpacked(held):
    """The codes of uint8 [..., D / 2], as float32 [..., D] less 8."""
    D = 2 * held.shape[-1]
    w = torch.stack((held & 15, held >> 4), -1).flatten(-2).unflatten(-1, (8, D // 32, 4))
    return w.transpose(-3, -2).flatten(-3).float() - 8.0


def _quantised(x, group):
    """Codes less 8 and scales of x [..., D] in 32 bits, one scale for `group` neighbouring values."""
    y = x.unflatten(-1, (-1, group))
    ratio = y.abs().amax(-1) / 7.0
    scale = ratio.to(torch.bfloat16)
    s = scale.float()[..., None]
    code = torch.sign(y) * torch.floor(y.abs() / torch.where(s > 0, s, 1.0) + 0.5)
    return code.flatten(-2), scale


def _pool(gen, pages, H, page, D, kind):
    """Cache contents as a program has them (codes or values, and scales) of normal values whose size varies."""
    held, scales = [], []
    for which in ("k", "v"):
        size = torch.exp(0.5 * torch.randn((pages, H, 1, 1), generator=gen, device="cuda"))
        x = torch.randn((pages, H, page, D), generator=gen, device="cuda") * size
        if kind == "bf16":
            held.append(x.to(torch.bfloat16))
            scales.append(None)
        elif kind == "e4m3":
            m, e = torch.frexp(x.abs().amax((2, 3)))  # the smallest power of two s with amax <= 448 s = 1.75 * 2^8 s
            s = torch.ldexp(torch.ones_like(m), torch.where(m <= 0.875, e - 9, e - 8))
            held.append((x / s[:, :, None, None]).to(torch.float8_e4m3fn))
            scales.append(s)
        else:
            code, s = _quantised(x, 32 if which == "k" else D)
            held.append(_packed(code + 8.0))
            scales.append(s if which == "k" else s[..., 0].contiguous())
    return dict(k_pool=held[0], v_pool=held[1], k_scale=scales[0], v_scale=scales[1])


def prepare(case, seed):
    gen = _generator(seed)
    op, D = case["op"], case["D"]
    if op == "prompt":
        new = _ragged(case["N"], case["longest"], case["ragged"])
        past = _past(case) if case["past"] else [0] * case["N"]
        keys = [n + p for n, p in zip(new, past)]

        def tokens(total, heads):
            if case["order"] == "thd":
                return _normal(gen, (1, total, heads, D), torch.bfloat16).transpose(1, 2)
            return _normal(gen, (1, heads, total, D), torch.bfloat16)

        q = tokens(sum(new), case["Hk"] * case["G"])
        k, v = (tokens(sum(keys), case["Hk"]) for _ in range(2))
        return _handles(dict(case=case, q=q, k=k, v=v, q_starts=_starts(new), k_starts=_starts(keys)))
    if op in ("store", "read"):
        H, page = case["H"], case["page"]
        new = _ragged(case["N"], case["longest"], case["ragged"])
        past = _past(case) if op == "store" else [0] * case["N"]
        lens = [n + p for n, p in zip(new, past)]
        table, pages = _page_table(gen, [-(-n // page) for n in lens], -(-max(lens) // page))
        s = dict(case=case, table=table, starts=_starts(lens), total=sum(lens),
                 **_pool(gen, pages, H, page, D, case.get("cache", "int4")))
        if op == "store":
            k, v = (_normal(gen, (1, sum(new), H, D), DTYPES[case["dtype"]]).transpose(1, 2) for _ in range(2))
            s.update(k=k, v=v, new_starts=_starts(new), past=torch.tensor(past, dtype=torch.int32, device="cuda"),
                     inv_freq=_inv_freq(case["rotary"]) if case["rotary"] else None)
        return _handles(s)
    B, H, page = case["B"], case["H"], case["page"]
    lens = _ragged(B, case["length"], case["ragged"])
    table, pages = _page_table(gen, [-(-n // page) for n in lens], -(-case["length"] // page))
    q = _normal(gen, (B, H * case["G"], case["Q"], D), torch.bfloat16)
    s = dict(case=case, q=q, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             **_pool(gen, pages, H, page, D, "int4"))
    if op == "step":
        k, v = (_normal(gen, (B, H, 1, D), torch.bfloat16) for _ in range(2))
        s.update(k=k, v=v, past=torch.tensor([max(n - 1, 0) for n in lens], dtype=torch.int32, device="cuda"),
                 new=torch.tensor([min(n, 1) for n in lens], dtype=torch.int32, device="cuda"),
                 inv_freq=_inv_freq(case["rotary"]) if case["rotary"] else None)
    return _handles(s)


def _handles(s):
    """What a program keeps between calls: the cache object, or the plan of a batch (one for all layers)."""
    if own:
        from block_sparse_masked_blockmask_gb300 import flexattn as fa
        c = s["case"]
        if c["op"] == "prompt":
            s["plan"] = fa.flex_packed_plan_create(s["q_starts"], s["k_starts"], s["q"].shape[2], s["k"].shape[2],
                                                   c["Hk"] * c["G"], c["Hk"], mask_kind=_mask_kind(fa, c),
                                                   window=c["window"], sinks=c["sinks"])
        else:
            s["kv"] = fa.KVCache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
    return s


def _mask_kind(fa, c):
    return fa.FLEX_MASK_WINDOW_SINKS if c["window"] else fa.FLEX_MASK_CAUSAL


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return {"prompt": _prompt, "store": _store, "read": _read, "step": _step, "cache": _cache}[state["case"]["op"]](state)


def _run_own(s):
    from block_sparse_masked_blockmask_gb300 import flexattn as fa
    c = s["case"]
    score = {"identity": fa.FLEX_SCORE_IDENTITY, "softcap": fa.FLEX_SCORE_SOFTCAP,
             "alibi": fa.FLEX_SCORE_ALIBI}[c.get("score", "identity")]
    layout = fa.FLEX_ROPE_INTERLEAVED if c.get("layout") == "interleaved" else fa.FLEX_ROPE_HALF
    if c["op"] == "prompt":
        return fa.flex_attention_packed_fwd(s["q"], s["k"], s["v"], s["plan"], score_kind=score, score_param=30.0)
    if c["op"] == "store":
        fa.flex_kv_cache_append_packed(s["kv"], s["k"], s["v"], s["new_starts"], s["table"], s["past"],
                                       inv_freq=s["inv_freq"], layout=layout)
    if c["op"] in ("store", "read"):
        return fa.flex_kv_cache_read(s["kv"], s["table"], s["starts"], s["total"], dtype=DTYPES[c["out"]])
    if c["op"] == "step":
        fa.flex_kv_cache_append(s["kv"], s["k"], s["v"], s["table"], s["past"], s["new"], inv_freq=s["inv_freq"],
                                layout=layout)
    out, lse = fa.flex_kv_cache_attention(s["q"], s["kv"], s["table"], s["lens"], mask_kind=_mask_kind(fa, c),
                                          window=c["window"], sinks=c["sinks"], score_kind=score, score_param=30.0)
    return (out, lse, s["k_scale"], s["v_scale"]) if c["op"] == "step" else (out, lse)


def _slopes(heads, dtype=torch.float32):
    return 2.0 ** (-8.0 * torch.arange(1, heads + 1, device="cuda", dtype=dtype) / heads)


def _scores(q, k, pos, c, heads):
    """Masked scores [Hk, G, rows, keys] of q [Hk, G, rows, D] at positions pos against k [Hk, keys, D]."""
    kv = torch.arange(k.shape[1], device="cuda")
    far = pos[:, None] - kv
    x = (q.flatten(1, 2) @ k.transpose(1, 2)).unflatten(1, q.shape[1:3]) / math.sqrt(q.shape[-1])
    if c["score"] == "softcap":
        x = 30.0 * torch.tanh(x / 30.0)
    elif c["score"] == "alibi":
        x = x - _slopes(heads).reshape(q.shape[0], q.shape[1], 1, 1) * far.float()
    keep = far >= 0
    if c["window"]:
        keep = keep & ((far < c["window"]) | (kv < c["sinks"]))
    return x.masked_fill(~keep, -math.inf)


def _softmax(x, v):
    """Rows of values and their lse, of scores [Hk, G, rows, keys] and v [Hk, keys, D]; nothing kept: 0 and -inf."""
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(1, 2) @ v).unflatten(1, x.shape[1:3])
    return torch.where(total > 0, out / total, 0.0), (top + total.log())[..., 0]


def _prompt(s):
    c = s["case"]
    Hk, G = c["Hk"], c["G"]
    q, k, v = s["q"][0], s["k"][0], s["v"][0]
    new = _ragged(c["N"], c["longest"], c["ragged"])
    past = _past(c) if c["past"] else [0] * c["N"]
    out = torch.empty_like(s["q"])
    lse = torch.empty((1, Hk * G, q.shape[1]), device="cuda")
    qa = ka = 0
    for n, p in zip(new, past):
        kb, vb = k[:, ka:ka + n + p].float(), v[:, ka:ka + n + p].float()
        rows = max(1, (1 << 29) // (Hk * G * max(1, n + p)))  # at most 2^29 scores at a time
        for a in range(0, n, rows):
            e = min(n, a + rows)
            seen = p + e  # later keys are masked for all of these rows
            x = _scores(q[:, qa + a:qa + e].float().unflatten(0, (Hk, G)), kb[:, :seen],
                        p + torch.arange(a, e, device="cuda"), c, Hk * G)
            o, l_ = _softmax(x, vb[:, :seen])
            out[0, :, qa + a:qa + e] = o.flatten(0, 1).to(out.dtype)
            lse[0, :, qa + a:qa + e] = l_.flatten(0, 1)
        qa, ka = qa + n, ka + n + p
    return out, lse


def _rotate(x, positions, inv_freq, layout):
    """x [H, tokens, D] in 32 bits, rotated by its positions [tokens]; the angles in 64."""
    angle = positions[:, None].double() * inv_freq
    cos, sin = angle.cos().float(), angle.sin().float()
    r = 2 * inv_freq.numel()
    part, rest = x[..., :r].float(), x[..., r:].float()
    if layout == "half":
        a, b = part[..., :r // 2], part[..., r // 2:]
        part = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((part, rest), -1)


def _write(s, k, v, b, pos):
    """Tokens k, v [H, tokens, D] of sequences b [tokens] at positions pos [tokens] into the 4-bit cache."""
    c, page = s["case"], s["case"]["page"]
    ids, at = s["table"][b, pos // page].long(), pos % page
    k = _rotate(k, pos, s["inv_freq"], c["layout"]) if s["inv_freq"] is not None else k.float()
    code, scale = _quantised(k.transpose(0, 1), 32)
    s["k_pool"][ids, :, at] = _packed(code + 8.0)
    s["k_scale"][ids, :, at] = scale
    code, scale = _quantised(v.float().transpose(0, 1), c["D"])
    s["v_pool"][ids, :, at] = _packed(code + 8.0)
    s["v_scale"][ids, :, at] = scale[..., 0]


def _places(starts, past, total):
    """Sequence and position of every packed token."""
    t = torch.arange(total, device="cuda")
    b = torch.searchsorted(starts[1:], t, right=True)
    return b, t - starts[b] + (past[b] if past is not None else 0)


def _held(s):
    """The values that the pools stand for, in 32 bits: keys, values [pages, H, page, D]."""
    k, v = s["k_pool"], s["v_pool"]
    if k.dtype == torch.bfloat16:
        return k.float(), v.float()
    if k.dtype == torch.float8_e4m3fn:
        return k.float() * s["k_scale"][:, :, None, None], v.float() * s["v_scale"][:, :, None, None]
    k = (_unpacked(k).unflatten(-1, (-1, 32)) * s["k_scale"].float()[..., None]).flatten(-2)
    return k, _unpacked(v) * s["v_scale"].float()[..., None]


def _store(s):
    b, pos = _places(s["new_starts"], s["past"], s["k"].shape[2])
    _write(s, s["k"][0], s["v"][0], b, pos)
    return _read(s)


def _read(s):
    c = s["case"]
    b, pos = _places(s["starts"], None, s["total"])
    ids, at = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    return tuple(x[ids, :, at].transpose(0, 1)[None].to(DTYPES[c["out"]]) for x in _held(s))


def _step(s):
    b = s["new"].nonzero()[:, 0]
    _write(s, s["k"][b, :, 0].transpose(0, 1), s["v"][b, :, 0].transpose(0, 1), b, s["past"][b].long())
    return _cache(s) + (s["k_scale"], s["v_scale"])


def _cache(s):
    c = s["case"]
    B, H, G, Q, D, page = c["B"], c["H"], c["G"], c["Q"], c["D"], c["page"]
    out = torch.empty_like(s["q"])
    lse = torch.empty((B, H * G, Q), device="cuda")
    ids = s["table"].clamp(min=0).long()
    few = max(1, (1 << 28) // (ids.shape[1] * page * H * D))  # sequences at a time: at most 2^28 values of the keys
    kv = torch.arange(ids.shape[1] * page, device="cuda")
    for a in range(0, B, few):
        e = min(B, a + few)
        held = dict(s, **{n: s[n][ids[a:e]].flatten(0, 1) for n in ("k_pool", "v_pool", "k_scale", "v_scale")})
        k, v = (x.unflatten(0, (e - a, -1)).transpose(1, 2).flatten(2, 3) for x in _held(held))  # [few, H, positions, D]
        x = s["q"][a:e].float().reshape(e - a, H, G * Q, D) @ k.transpose(2, 3) / math.sqrt(D)
        pos = s["lens"][a:e, None] - Q + torch.arange(Q, device="cuda")
        far = (pos[:, :, None] - kv).repeat(1, G, 1)[:, None]                         # rows: G heads of Q tokens
        if c["score"] == "softcap":
            x = 30.0 * torch.tanh(x / 30.0)
        elif c["score"] == "alibi":
            x = x - _slopes(H * G).reshape(1, H, G, 1).repeat_interleave(Q, 2) * far.float()
        keep = far >= 0
        if c["window"]:
            keep = keep & ((far < c["window"]) | (kv < c["sinks"]))
        x = x.masked_fill(~keep, -math.inf)
        top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
        p = (x - top).exp()
        total = p.sum(-1, keepdim=True)
        v = v.masked_fill((kv >= s["lens"][a:e, None])[:, None, :, None], 0.0)         # what lies behind the last token
        o = torch.where(total > 0, (p @ v) / total, 0.0)
        out[a:e] = o.reshape(e - a, H * G, Q, D).to(out.dtype)
        lse[a:e] = (top + total.log()).reshape(e - a, H * G, Q)
    return out, lse


# ----------------------------------------------------------------- the work
def _pairs(n, p, W, sinks):
    """(row, key) pairs of n rows at positions p .. p + n - 1, and the keys that some row sees."""
    if not W:
        return n * p + n * (n + 1) // 2, p + n if n else 0
    pairs = sum(min(i + 1, W + min(sinks, max(0, i + 1 - W))) for i in range(p, p + n))
    low = max(0, p - W + 1)
    return pairs, p + n - low + min(sinks, low) if n else 0


def _token_bytes(D, kind):
    """Bytes of a key and a value of one head, their scales with them."""
    return {"int4": D + D / 16 + 2, "e4m3": 2 * D, "bf16": 4 * D}[kind]


def work(case):
    op, D = case["op"], case["D"]
    if op == "prompt":
        new = _ragged(case["N"], case["longest"], case["ragged"])
        past = _past(case) if case["past"] else [0] * case["N"]
        heads = case["Hk"] * case["G"]
        pairs, seen = (sum(x) for x in zip(*(_pairs(n, p, case["window"], case["sinks"]) for n, p in zip(new, past))))
        return {"bytes": 4.0 * seen * case["Hk"] * D + sum(new) * heads * (4.0 * D + 4), "flops": 4.0 * pairs * heads * D}
    if op in ("store", "read"):
        new = sum(_ragged(case["N"], case["longest"], case["ragged"]))
        size = 2 if case["out"] == "bf16" else 4
        if op == "read":
            n = new * case["H"]
            return {"bytes": n * (_token_bytes(D, case["cache"]) + 2.0 * D * size), "flops": 2.0 * n * D}
        total = (new + sum(_past(case))) * case["H"]
        held, src = _token_bytes(D, "int4"), 2 if case["dtype"] == "bf16" else 4
        return {"bytes": new * case["H"] * (2.0 * D * src + held) + total * (held + 2.0 * D * size),
                "flops": 2.0 * total * D + 8.0 * new * case["H"] * D}
    heads, Q = case["H"] * case["G"], case["Q"]
    pairs = seen = rows = 0
    for n in _ragged(case["B"], case["length"], case["ragged"]):
        q = min(n, Q)
        a, b = _pairs(q, n - q, case["window"], case["sinks"])
        pairs, seen, rows = pairs + a, seen + b, rows + q
    held = _token_bytes(D, "int4")
    step = rows * case["H"] * (4.0 * D + held) if op == "step" else 0.0
    return {"bytes": seen * case["H"] * held + case["B"] * Q * heads * (4.0 * D + 4) + step,
            "flops": 4.0 * pairs * heads * D}


# ---------------------------------------------------------- in 64 bits, apart
def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "store": _exact_store, "read": _exact_read, "step": _exact_step,
            "cache": _exact_cache}[case["op"]](s)


def _exact_rows(q, k, v, pos, c):
    """q [heads, rows, D] at positions pos (a list's tensor) against k, v [Hk, keys, D], all float64."""
    heads, _, D = q.shape
    kv = torch.arange(k.shape[1], device="cuda")
    hidden = kv[None] > pos[:, None]
    if c["window"]:
        hidden |= (pos[:, None] - kv >= c["window"]) & (kv >= c["sinks"])
    group = heads // k.shape[0]
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    live = ~hidden.all(1)
    if not bool(live.any()):
        return out, lse
    slope = _slopes(heads, torch.float64)
    for h in range(heads):
        x = torch.einsum("rd,kd->rk", q[h], k[h // group]) * D ** -0.5
        if c["score"] == "softcap":
            x = 30.0 * torch.tanh(x / 30.0)
        elif c["score"] == "alibi":
            x = x - slope[h] * (pos[:, None] - kv).double()
        x.masked_fill_(hidden, -math.inf)
        lse[h] = torch.logsumexp(x, -1)
        out[h] = torch.einsum("rk,kd->rd", torch.where(live[:, None], torch.softmax(x, -1), 0.0), v[h // group])
    return out, lse


def _exact_prompt(s):
    c = s["case"]
    q, k, v = s["q"][0].double(), s["k"][0].double(), s["v"][0].double()
    new = _ragged(c["N"], c["longest"], c["ragged"])
    past = _past(c) if c["past"] else [0] * c["N"]
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    qa = ka = 0
    for n, p in zip(new, past):
        for a in range(0, n, 2048):
            e = min(a + 2048, n)
            out[:, qa + a:qa + e], lse[:, qa + a:qa + e] = _exact_rows(
                q[:, qa + a:qa + e], k[:, ka:ka + p + e], v[:, ka:ka + p + e], torch.arange(p + a, p + e, device="cuda"), c)
        qa, ka = qa + n, ka + n + p
    return out[None], lse[None]


def _exact_quantised(x, group):
    """The values that x [..., D] in 64 bits is held as in 4 bits, and their scales."""
    y = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    step = (y.abs().amax(-1, keepdim=True) / 7.0).to(torch.bfloat16).double()
    n = torch.where(step > 0, torch.floor(y.abs() / step + 0.5), torch.zeros_like(y))
    return (torch.copysign(n, y) * step).reshape(x.shape), step[..., 0]


def _turned(x, pos, inv_freq, layout):
    """Complex form of the rotation: (x0 + i x1) exp(i position freq), of x [tokens, H, D]."""
    r = 2 * inv_freq.numel()
    y = x.double().clone()
    first, second = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    angle = pos.double()[:, None, None] * inv_freq
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(angle), angle)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_held(s, b, n):
    """Keys and values of sequence b's first n tokens in 64 bits [n, H, D], value by value from the pools."""
    c = s["case"]
    D, page = c["D"], c["page"]
    t = torch.arange(n, device="cuda")
    ids = s["table"][b].long()[t // page]
    results = []
    for pool, scale in ((s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"])):
        rows = pool[ids, :, t % page]
        if pool.dtype != torch.uint8:
            x = rows.double()
            results.append(x if scale is None else x * scale[ids].double()[..., None])
            continue
        d = torch.arange(D, device="cuda")
        word = (D // 32) * (d % 32 // 4) + d // 32
        byte, high = 2 * word + d % 4 // 2, d % 2
        code = (rows[..., byte].int() >> (4 * high)) & 15
        sc = scale[ids, :, t % page].double()
        sc = sc[..., d // 32] if sc.dim() == 3 else sc[..., None]
        results.append((code.double() - 8) * sc)
    return results


def _exact_new(s, k, v, pos):
    """New tokens k, v [tokens, H, D] at positions pos, as the 4-bit cache holds them: (values, scales) of each."""
    k = _turned(k, pos, s["inv_freq"], s["case"]["layout"]) if s["inv_freq"] is not None else k.double()
    return _exact_quantised(k, 32), _exact_quantised(v.double(), s["case"]["D"])


def _exact_store(s):
    c = s["case"]
    new, past, at = _ragged(c["N"], c["longest"], c["ragged"]), _past(c), 0
    ks, vs = [], []
    for b, (n, p) in enumerate(zip(new, past)):
        k, v = _exact_held(s, b, p)
        (kn, _), (vn, _) = _exact_new(s, s["k"][0, :, at:at + n].transpose(0, 1),
                                      s["v"][0, :, at:at + n].transpose(0, 1), torch.arange(p, p + n, device="cuda"))
        ks += [k, kn]
        vs += [v, vn]
        at += n
    return tuple(torch.cat(x).transpose(0, 1)[None] for x in (ks, vs))


def _exact_read(s):
    c = s["case"]
    held = [_exact_held(s, b, n) for b, n in enumerate(_ragged(c["N"], c["longest"], c["ragged"]))]
    return tuple(torch.cat(x).transpose(0, 1)[None] for x in zip(*held))


def _exact_step(s):
    return _exact_cache(s) + (s["k_scale"].double(), s["v_scale"].double())


def _exact_cache(s):
    c = s["case"]
    H, G, Q, D = c["H"], c["G"], c["Q"], c["D"]
    out = torch.zeros((c["B"], H * G, Q, D), dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], H * G, Q), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_ragged(c["B"], c["length"], c["ragged"])):
        if not n:
            continue
        k, v = _exact_held(s, b, n)
        if c["op"] == "step":
            (k[n - 1:], ks), (v[n - 1:], vs) = _exact_new(s, s["k"][b].transpose(0, 1), s["v"][b].transpose(0, 1),
                                                          torch.tensor([n - 1], device="cuda"))
            pid, at = int(s["table"][b, (n - 1) // c["page"]]), (n - 1) % c["page"]
            s["k_scale"][pid, :, at], s["v_scale"][pid, :, at] = ks[0].to(torch.bfloat16), vs[0, :, 0].to(torch.bfloat16)
        out[b], lse[b] = _exact_rows(s["q"][b].double(), k.transpose(0, 1), v.transpose(0, 1),
                                     torch.arange(n - Q, n, device="cuda"), c)
    return out, lse
