"""Cases of the operators around a paged cache: what turns queries and keys to
their positions, what holds keys and values in 4 bits, and the attention that
reads them there.

    rotate  rotary positions, and their gradient
    store   keys and values quantised into their slots, and read back
    attend  attention over the cache, from single tokens to prompts

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is true, by the calls of ``Tokenizer``.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
GROUP = 32  # elements that share a step and a base


def listed():
    return [
        # one decode step of a small batch: queries and keys of a fused projection
        {"name": "rotate, 8 tokens", "op": "rotate", "tokens": 8, "heads": 40, "dim": 128, "part": 128,
         "interleaved": False, "factor": 1.0, "far": 4000, "type": "bf16", "grad": False},
        # prompts of a model that turns a part of each head, scaled to contexts of 131072; odd sizes
        {"name": "rotate, 5003 tokens, 50 of 80", "op": "rotate", "tokens": 5003, "heads": 21, "dim": 80, "part": 50,
         "interleaved": True, "factor": 16.0, "far": 131_072, "type": "f16", "grad": False},
        # a training batch, forward and backward
        {"name": "rotate, 65536 tokens and gradient", "op": "rotate", "tokens": 65_536, "heads": 40, "dim": 128,
         "part": 128, "interleaved": False, "factor": 1.0, "far": 8192, "type": "bf16", "grad": True},
        # the keys and values of a decode step
        {"name": "store, 8 tokens", "op": "store", "tokens": 8, "heads": 8, "dim": 128, "block": 16, "type": "bf16"},
        # prompts of a small model in half precision, an odd head and blocks of 100
        {"name": "store, 9001 tokens, dim 72", "op": "store", "tokens": 9001, "heads": 5, "dim": 72, "block": 100,
         "type": "f16"},
        # the prompts of a large batch
        {"name": "store, 131072 tokens", "op": "store", "tokens": 131_072, "heads": 8, "dim": 128, "block": 16,
         "type": "bf16"},
        # a few requests of an interactive server, one new token each
        {"name": "attend, 8 requests", "op": "attend", "requests": 8, "new": 0, "cached": 4000, "heads": 8, "group": 4,
         "dim": 128, "block": 16, "type": "bf16"},
        # one request over a long document
        {"name": "attend, 1 request of 131072", "op": "attend", "requests": 1, "new": 0, "cached": 131_072,
         "heads": 8, "group": 5, "dim": 128, "block": 64, "type": "bf16"},
        # a large running batch
        {"name": "attend, 384 requests", "op": "attend", "requests": 384, "new": 0, "cached": 4000, "heads": 8,
         "group": 8, "dim": 128, "block": 16, "type": "bf16"},
        # drafted tokens of running requests are checked, a model in half precision with small heads
        {"name": "attend, 100 requests, drafts", "op": "attend", "requests": 100, "new": 500, "cached": 1500,
         "heads": 6, "group": 3, "dim": 64, "block": 32, "type": "f16"},
        # a model in 32 bits without shared heads, wide and odd ones, odd blocks
        {"name": "attend, 5 requests f32, dim 200", "op": "attend", "requests": 5, "new": 0, "cached": 700, "heads": 7,
         "group": 1, "dim": 200, "block": 7, "type": "f32"},
        # a step with chunks of prompts behind what is cached
        {"name": "attend, 16 prompts", "op": "attend", "requests": 16, "new": 8000, "cached": 3000, "heads": 8,
         "group": 4, "dim": 128, "block": 16, "type": "bf16"},
    ]


#: Bytes and operations of one pass that a drawn case of an operator does not pass.
MOST_BYTES = {"rotate": 2_600_000_000, "store": 1_350_000_000, "attend": 1_900_000_000}
MOST_FLOPS = {"rotate": 1e15, "store": 1e15, "attend": 4e11}
MOST_SCORES = 1_500_000_000  # of queries and tokens: the plain form holds those of a request at once


def draw(rng):
    def span(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rotate", "store", "attend", "attend"])
    dim = rng.choice([64, 128, 32 * span(1, 8), 8 * span(2, 32), span(16, 256)])
    kind = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op == "rotate":
        dim += dim % 2
        part = rng.choice([dim, dim, 2 * rng.randint(1, dim // 2)])
        c = {"op": op, "tokens": span(1, 131_072), "heads": span(1, 80), "dim": dim, "part": part,
             "interleaved": rng.random() < 0.5, "factor": rng.choice([1.0, 4.0, 32.0]),
             "far": span(100, 1_000_000), "type": kind, "grad": rng.random() < 0.4}
        shrink = ("tokens",)
    elif op == "store":
        c = {"op": op, "tokens": span(1, 200_000), "heads": span(1, 32), "dim": dim,
             "block": rng.choice([1, 8, 16, 16, 32, 64, 100, 128, 256]), "type": kind}
        shrink = ("tokens",)
    else:
        n = span(1, 384)
        c = {"op": op, "requests": n, "new": rng.choice([0, 0, 1]) * (n + span(1, 8000)), "cached": span(1, 131_072),
             "heads": span(1, 16), "group": rng.choice([1, 2, 3, 4, 8, span(1, 16)]), "dim": dim,
             "block": rng.choice([1, 8, 16, 16, 32, 64, 100, 128, 256]), "type": kind}
        shrink = ("cached", "new")
    most = MOST_FLOPS[op] if op != "attend" else min(MOST_FLOPS[op], 4 * dim * MOST_SCORES)
    while work(c)["bytes"] > MOST_BYTES[op] or work(c)["flops"] > most:
        for key in shrink:
            c[key] = c[key] * 7 // 8
        if c.get("new"):
            c["new"] = max(c["new"], c["requests"])
    return c


# ------------------------------------------------------------------ inputs --

def _frequencies(part, factor):
    """Radians a position of each pair: base 10000, beyond 8192 positions by
    parts, from 1 turn over the trained length (stretched whole) to 4 (kept)."""
    f = 10_000.0 ** (-np.arange(0, part, 2, dtype=np.float64) / part)
    if factor != 1.0:
        keep = np.clip((8192 * f / (2 * np.pi) - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    return f


def _groups(dim):
    """Groups of a row in the cache: an even number beyond four."""
    g = (dim + GROUP - 1) // GROUP
    return g + g % 2 if g > 4 else g


def _page_bytes(block, dim):
    """Of one head in one block: the codes of its rows, then their steps and bases, to whole 16 bytes."""
    return (block * _groups(dim) * 20 + 15) // 16 * 16


def _code_order(dim):
    """The element of each of a row's codes, low half of a byte first: pairs of
    groups share 32 bytes, their words of 8 codes in turn; a last group without
    a partner is in order."""
    g = _groups(dim)
    at = np.arange(g * GROUP)
    unit, rest = at // 64, at % 64
    mixed = unit * 64 + rest % 16 // 8 * 32 + rest // 16 * 8 + rest % 8
    return np.where(at < g // 2 * 64, mixed, at)


def _lens(case):
    """Tokens of each request after the step, new ones among them: from next to nothing to twice the mean."""
    n = case["requests"]
    spread = (np.arange(n) + 0.5) * 2 / n if n > 1 else np.ones(1)
    return np.maximum((spread * case["cached"]).astype(np.int64), 0)


def _new(case):
    """New tokens of each request; prompts of very different lengths."""
    n = case["requests"]
    if not case["new"]:
        return np.ones(n, dtype=np.int64)
    share = (np.arange(n) * 7 % n + 1.0) ** (2 if case["new"] > 20 * n else 1)
    new = np.maximum((share / share.sum() * case["new"]).astype(np.int64), 1)
    while new.sum() > case["new"]:
        new[new.argmax()] -= 1
    return new


_program = {}


def _tokenizer():
    """The handle that a program keeps: one tokenizer, here of the 256 bytes alone."""
    if "tok" not in _program:
        import byte_level_bpe_pretokenize_gb300 as bpe
        _program["tok"] = bpe.Tokenizer(np.zeros((0, 3), np.int32), np.arange(256, dtype=np.uint8),
                                        np.arange(257, dtype=np.int64))
    return _program["tok"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if own:
        s["tok"] = _tokenizer()  # the same inputs on either side
    op, dim = case["op"], case["dim"]
    dtype = TYPES[case["type"]]

    def normal(*shape, by=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * by).to(dtype)

    if op == "rotate":
        shape = (case["tokens"], case["heads"], dim)
        s["x"] = normal(*shape)
        s["positions"] = torch.randint(0, case["far"], shape[:1], generator=gen, device="cuda", dtype=torch.int32)
        s["frequencies"] = _frequencies(case["part"], case["factor"])
        s["magnitude"] = 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0
        if own:
            s["table"] = s["tok"].rotary_table(case["part"], base=10_000.0, factor=case["factor"], original=8192,
                                               low=1.0, high=4.0)
        if case["grad"]:
            s["upstream"] = normal(*shape)
        return s
    heads, block = case["heads"], case["block"]
    row = _groups(dim) * 16
    if op == "store":
        n = case["tokens"]
        blocks = (n + block - 1) // block + 3
        s["cache"] = torch.zeros(blocks, 2, heads, _page_bytes(block, dim), dtype=torch.uint8, device="cuda")
        # keys differ from channel to channel, with a few far out; a padded step has tokens without a slot
        away = torch.randn(heads, dim, generator=gen, device="cuda")
        away += (torch.rand(heads, dim, generator=gen, device="cuda") < 0.02) * 12.0
        s["keys"] = (torch.randn(n, heads, dim, generator=gen, device="cuda") + away).to(dtype)
        s["values"] = normal(n, heads, dim, by=0.7)
        slots = torch.randperm(blocks * block, generator=gen, device="cuda")[:n].sort().values
        if n > 8:
            slots[-(n // 50 + 1):] = -1
        s["slots"] = slots
        return s
    n = case["requests"]
    new = _new(case)
    lens = _lens(case) + new
    shuffle = torch.randperm(n, generator=gen, device="cuda").cpu().numpy()
    new, lens = new[shuffle], lens[shuffle]
    s["new_host"], s["lens_host"] = new.tolist(), lens.tolist()
    held = (lens + block - 1) // block
    blocks = int(held.sum()) + 2
    s["cache"] = torch.randint(0, 256, (blocks, 2, heads, _page_bytes(block, dim)), generator=gen, device="cuda",
                               dtype=torch.uint8)
    # steps and bases of rows whose values are about normal; the last groups' padding has codes too
    pairs = s["cache"].view(torch.bfloat16)[..., block * row // 2:block * row // 2 + block * row // 8]
    step = torch.rand(*pairs.shape[:-1], pairs.shape[-1] // 2, generator=gen, device="cuda") * 0.2 + 0.15
    pairs[..., 1::2] = (-8 * step + 0.3 * torch.randn(step.shape, generator=gen, device="cuda")).to(torch.bfloat16)
    pairs[..., 0::2] = step.to(torch.bfloat16)
    width = int(held.max()) + 1
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    there = torch.arange(width, device="cuda")[None, :] < torch.from_numpy(held).cuda()[:, None]
    table[there] = torch.randperm(blocks, generator=gen, device="cuda")[:int(held.sum())].to(torch.int32)
    s["block_table"] = table
    s["seq_lens"] = torch.from_numpy(lens).to(torch.int32).cuda()
    s["offsets"] = None
    if case["new"]:
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).cuda()
    s["queries"] = normal(int(new.sum()), heads * case["group"], dim, by=1.5)
    return s


# -------------------------------------------------------------------- pass --

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_rotate(s):
    tok = s["tok"]
    if not s["grad"]:
        return tok.rotate(s["x"], s["positions"], s["table"], interleaved=s["interleaved"], scale=s["magnitude"])
    x = s["x"].detach().requires_grad_()
    y = tok.rotate(x, s["positions"], s["table"], interleaved=s["interleaved"], scale=s["magnitude"])
    (grad,) = torch.autograd.grad(y, x, s["upstream"])
    return y.detach(), grad


def _own_store(s):
    s["tok"].write_cache(s["cache"], s["slots"], s["keys"], s["values"], s["block"])
    return s["tok"].read_cache(s["cache"], s["slots"], s["dim"], s["block"], dtype=TYPES[s["type"]])


def _own_attend(s):
    return s["tok"].attend(s["queries"], s["cache"], s["block_table"], s["seq_lens"], s["block"],
                           offsets=s["offsets"])


_own = {"rotate": _own_rotate, "store": _own_store, "attend": _own_attend}


def _turn(x, cos, sin, part, interleaved):
    """x [tokens, heads, dim] turned, in 32 bits and rounded to x's type."""
    y = x.float()
    a, b = (y[..., 0:part:2], y[..., 1:part:2]) if interleaved else (y[..., :part // 2], y[..., part // 2:part])
    c, d = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([turned, y[..., part:]], -1).to(x.dtype)


def _plain_rotate(s):
    # far positions: the angle in 64 bits
    angle = s["positions"].double()[:, None] * torch.from_numpy(s["frequencies"]).cuda()
    cos, sin = ((f(angle) * s["magnitude"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    y = _turn(s["x"], cos, sin, s["part"], s["interleaved"])
    if not s["grad"]:
        return y
    return y, _turn(s["upstream"], cos, -sin, s["part"], s["interleaved"])


def _plain_store(s):
    dim, block, cache, slots = s["dim"], s["block"], s["cache"], s["slots"]
    groups = _groups(dim)
    row = groups * 16
    order = torch.from_numpy(_code_order(dim)).cuda()
    there = slots >= 0
    at = slots[there]
    page, place = at // block, at % block
    n, heads = at.numel(), s["heads"]
    out = []
    for which, x in enumerate((s["keys"], s["values"])):
        x = torch.nn.functional.pad(x[there].float(), (0, groups * GROUP - dim), value=math.nan)
        x = x.reshape(n, heads, groups, GROUP)
        hole = x.isnan()
        low, high = (torch.where(hole, -f, x).amin(-1) if f < 0 else torch.where(hole, -f, x).amax(-1)
                     for f in (-math.inf, math.inf))
        low, high = (torch.where(t.isinf(), 0.0, t) for t in (low, high))
        base = low.to(torch.bfloat16).float()
        step = ((high * 0.5 - base * 0.5) / 7.5).clamp(min=0).to(torch.bfloat16).float()
        step = torch.where(step < 2.0 ** -100, 0.0, step)
        by = torch.where(step > 0, 1.0 / (step * 0.5), 0.0)
        code = ((x * 0.5 - base[..., None] * 0.5) * by[..., None]).round().clamp(0, 15)
        code = torch.where(hole, 0.0, code).to(torch.uint8).reshape(n, heads, -1)[..., order]
        rows = cache[:, which, :, :block * row].unflatten(-1, (block, row))
        rows[page, :, place] = code[..., 0::2] | code[..., 1::2] << 4
        pair = torch.stack([step, base], -1).to(torch.bfloat16).flatten(-2).view(torch.uint8)
        pairs = cache[:, which, :, block * row:block * row * 5 // 4].unflatten(-1, (block, row // 4))
        pairs[page, :, place] = pair
        # and back
        y = torch.zeros(slots.numel(), heads, dim, dtype=x.dtype, device="cuda")
        y[there] = _values(rows[page, :, place], pairs[page, :, place], dim, order)
        out.append(y.to(TYPES[s["type"]]))
    return tuple(out)


def _values(codes, pairs, dim, order):
    """What rows of codes and of (step, base) pairs stand for, in 32 bits."""
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    back = torch.empty_like(code)
    back[..., order] = code
    pair = pairs.contiguous().view(torch.bfloat16).float()
    value = back.unflatten(-1, (-1, GROUP)) * pair[..., 0::2, None] + pair[..., 1::2, None]
    return value.flatten(-2)[..., :dim]


def _plain_attend(s):
    dim, block, heads, group, cache = s["dim"], s["block"], s["heads"], s["group"], s["cache"]
    row = _groups(dim) * 16
    order = torch.from_numpy(_code_order(dim)).cuda()
    n, q = s["requests"], s["queries"]
    lens, new = s["lens_host"], s["new_host"]
    starts = np.concatenate([[0], np.cumsum(new)])
    out = torch.empty_like(q)
    i = 0
    while i < n:
        # as many requests at a time as have room, padded to the longest
        j, most, longest = i, 0, 0
        while j < n and (j == i or (j + 1 - i) * heads * max(longest, lens[j]) *
                         (dim + group * max(most, new[j])) < 2 ** 28):
            longest, most = max(longest, lens[j]), max(most, new[j])
            j += 1
        pages = s["block_table"][i:j, :(longest + block - 1) // block].clamp(min=0).long()
        kv = []
        for which in (0, 1):
            page = cache[pages, which]  # [requests, pages, heads, bytes]
            codes = page[..., :block * row].unflatten(-1, (block, row)).transpose(1, 2).flatten(2, 3)
            pairs = page[..., block * row:block * row * 5 // 4].unflatten(-1, (block, row // 4))
            pairs = pairs.transpose(1, 2).flatten(2, 3)
            kv.append(_values(codes[:, :, :longest], pairs[:, :, :longest], dim, order))
        k, v = kv
        at = torch.arange(most, device="cuda")
        m = torch.tensor(new[i:j], device="cuda")[:, None]
        src = torch.tensor(starts[i:j].tolist(), device="cuda")[:, None] + at
        real = at < m
        x = q[torch.where(real, src, 0)].float()  # [requests, new, heads * group, dim]
        x = x.unflatten(2, (heads, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
        score = x @ k.transpose(-1, -2) * dim ** -0.5
        upto = torch.tensor(lens[i:j], device="cuda")[:, None] - m + at
        seen = torch.arange(longest, device="cuda") <= upto[..., None]  # [requests, new, tokens]
        score = score.unflatten(2, (most, group)).masked_fill(~seen[:, None, :, None], -math.inf)
        top = score.amax(-1, keepdim=True)
        p = torch.exp(score - top)
        y = (p / p.sum(-1, keepdim=True)).flatten(2, 3) @ v
        y = y.unflatten(2, (most, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
        out[src[real]] = y[real].to(out.dtype)
        i = j
    return out


_plain = {"rotate": _plain_rotate, "store": _plain_store, "attend": _plain_attend}


# ----------------------------------------------------------- what it needs --

def work(case):
    op, dim, size = case["op"], case["dim"], SIZE[case["type"]]
    if op == "rotate":
        passes = 2 if case["grad"] else 1
        n = case["tokens"] * case["heads"]
        return {"bytes": passes * (2 * n * dim * size + 4 * case["tokens"]), "flops": passes * 3 * n * case["part"]}
    held = dim / 2 + 4 * math.ceil(dim / GROUP)  # of a key or a value
    heads = case["heads"]
    if op == "store":
        rows = 2 * case["tokens"] * heads
        return {"bytes": rows * (2 * dim * size + 2 * held) + 16 * case["tokens"], "flops": 5 * rows * dim}
    new = _new(case).astype(np.float64)
    lens = _lens(case) + new
    pairs = float((new * lens - new * (new - 1) / 2).sum())  # of a new token and one that it sees
    rows = float(lens.sum()) * heads * 2
    return {"bytes": rows * held + 2 * float(new.sum()) * heads * case["group"] * dim * size + 8 * case["requests"]
            + 4 * float(lens.sum()) / case["block"], "flops": 4 * pairs * heads * case["group"] * dim}


def exact(case, seed):
    s = prepare(case, seed)
    op, dim = case["op"], case["dim"]
    if op == "rotate":
        half = case["part"] // 2
        first = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        angle = s["positions"].double().outer(torch.from_numpy(s["frequencies"]).cuda())[:, None, :]
        z = torch.polar(torch.full_like(angle, s["magnitude"]), angle)
        out = []
        for x, turn in ((s["x"], z),) + (((s["upstream"], z.conj()),) if case["grad"] else ()):
            y = x.double()
            w = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = w.real, w.imag
            out.append(y)
        return tuple(out) if case["grad"] else out[0]
    if op == "store":
        # the definition is in 32 bits, rounding by rounding
        slots = s["slots"].cpu().numpy()
        out = []
        for x in (s["keys"], s["values"]):
            x = x.float().cpu().numpy()
            y = np.zeros(x.shape)
            for lo in range(0, dim, GROUP):
                g = x[..., lo:lo + GROUP]
                base = _bf16(g.min(-1))
                step = np.maximum(_bf16((np.float32(0.5) * g.max(-1) - np.float32(0.5) * base) / np.float32(7.5)), 0)
                step[step < 2.0 ** -100] = 0
                with np.errstate(divide="ignore"):
                    by = np.where(step > 0, np.float32(1) / (np.float32(0.5) * step), 0).astype(np.float32)
                code = (np.float32(0.5) * g - np.float32(0.5) * base[..., None]) * by[..., None]
                code = np.clip(np.rint(code), 0, 15)
                y[..., lo:lo + GROUP] = base[..., None].astype(np.float64) + step[..., None] * code.astype(np.float64)
            y[slots < 0] = 0
            out.append(torch.from_numpy(y))
        return tuple(out)
    # attend: a request and a head at a time
    block, heads, group = case["block"], case["heads"], case["group"]
    if work(case)["bytes"] * heads > 4e10:
        return None
    units = _groups(dim)
    where = np.empty(units * GROUP, dtype=np.int64)  # the place of each element's code
    for e in range(units * GROUP):
        g, i = divmod(e, GROUP)
        alone = units % 2 == 1 and g == units - 1
        where[e] = e if alone else g // 2 * 64 + (i // 8 * 2 + g % 2) * 8 + i % 8
    where = torch.from_numpy(where).cuda()[:dim]
    share = torch.arange(dim, device="cuda") // GROUP
    out = torch.zeros(s["queries"].shape, dtype=torch.float64, device="cuda")
    start = 0
    for r, (length, new) in enumerate(zip(s["lens_host"], s["new_host"])):
        t = torch.arange(length, device="cuda")
        page, place = s["block_table"][r, t // block].long(), t % block
        for h in range(heads):
            kv = []
            for which in (0, 1):
                flat = s["cache"][:, which, h]
                byte = flat[page[:, None], place[:, None] * units * 16 + where // 2].long()
                code = (byte >> (where % 2 * 4)) & 15
                at = block * units * 16 + (place[:, None] * units + share) * 4
                bits = [flat[page[:, None], at + k].int() for k in range(4)]
                step, base = ((lo << 16 | hi << 24).view(torch.float32).double() for lo, hi in (bits[:2], bits[2:]))
                kv.append(base + step * code)
            x = s["queries"][start:start + new, h * group:(h + 1) * group].double()
            score = torch.einsum("qgd,td->qgt", x, kv[0]) / math.sqrt(dim)
            last = length - new + torch.arange(new, device="cuda")
            score[(t[None, :] > last[:, None])[:, None, :].expand_as(score)] = -math.inf
            out[start:start + new, h * group:(h + 1) * group] = torch.einsum("qgt,td->qgd", score.softmax(-1), kv[1])
        start += new
    return out


def _bf16(x):
    """float32 rounded to the nearest bfloat16, ties to even."""
    bits = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    bits = (bits + 0x7FFF + (bits >> 16 & 1)) & 0xFFFF0000
    return bits.astype(np.uint32).view(np.float32)
