"""Cases of the operators around the encoder: what carries its packed ids into a
language model and what prepares the model's logits for the next ids.

    plan    block tables, slots and positions of a batch of requests
    embed   the rows of an embedding table, scaled
    grad    the embedding table's gradient
    logits  penalties for repeated tokens, biases and grammar masks

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
#: Bytes of one pass that a drawn case of an operator does not pass.
MOST = {"plan": 19_000_000, "embed": 700_000_000, "grad": 1_100_000_000, "logits": 180_000_000}


def listed():
    return [
        # a few requests of an interactive server, one new token each
        {"name": "plan, 8 single tokens", "op": "plan", "requests": 8, "tokens": 0, "cached": 4000, "block": 16,
         "free": 1.0, "pad": 0},
        # a step that mixes running requests with chunks of prompts, padded for a captured graph; the cache runs short
        {"name": "plan, 500 requests, short", "op": "plan", "requests": 500, "tokens": 8000, "cached": 9000,
         "block": 32, "free": 0.8, "pad": 192},
        # the prompts of a whole batch of documents (as many as the mixed-script workload has)
        {"name": "plan, 16384 prompts", "op": "plan", "requests": 16384, "tokens": 1_500_001, "cached": 60,
         "block": 16, "free": 1.0, "pad": 63},
        # one decode step of a small batch
        {"name": "embed, 8 tokens", "op": "embed", "tokens": 8, "rows": 69_424, "dim": 2048, "weight": "bf16",
         "out": "bf16", "scale": 1.0},
        # prompts of a server in half precision, a width that 8 does not divide
        {"name": "embed, 5003 tokens, dim 1234", "op": "embed", "tokens": 5003, "rows": 32_256, "dim": 1234,
         "weight": "f16", "out": "f16", "scale": 35.125},
        # a training batch: master weights in 32 bits, activations in bfloat16
        {"name": "embed, 65536 tokens", "op": "embed", "tokens": 65_536, "rows": 69_424, "dim": 4096,
         "weight": "f32", "out": "bf16", "scale": 64.0},
        # fine-tuning on one short document with the smallest table
        {"name": "grad, 300 tokens", "op": "grad", "tokens": 300, "rows": 768, "dim": 512, "grad": "f32",
         "weight": "f32", "scale": 1.0},
        # a micro-batch of a small model, odd sizes
        {"name": "grad, 9001 tokens, dim 777", "op": "grad", "tokens": 9001, "rows": 32_256, "dim": 777,
         "grad": "f16", "weight": "f32", "scale": 27.875},
        # a training batch with bfloat16 activations and gradients
        {"name": "grad, 65536 tokens", "op": "grad", "tokens": 65_536, "rows": 69_424, "dim": 4096, "grad": "bf16",
         "weight": "bf16", "scale": 64.0},
        # one request, its prompt against repetition
        {"name": "logits, 1 request", "op": "logits", "requests": 1, "vocab": 32_256, "prompt": 200, "output": 60,
         "bias": 0, "masks": 0.0, "logits": "f32", "out": "f32"},
        # a running batch: penalties, a few biases, a grammar for half of the requests, 32 bits for the sampler
        {"name": "logits, 48 requests", "op": "logits", "requests": 48, "vocab": 69_424, "prompt": 1200,
         "output": 400, "bias": 40, "masks": 0.5, "logits": "bf16", "out": "f32"},
        # a large batch with long prompts, an odd vocabulary and a grammar for each request
        {"name": "logits, 384 requests", "op": "logits", "requests": 384, "vocab": 113_645, "prompt": 3000,
         "output": 900, "bias": 10, "masks": 1.0, "logits": "bf16", "out": "bf16"},
    ]


def draw(rng):
    def span(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["plan", "embed", "grad", "logits"])
    rows = rng.choice([768, 32_256, 69_424, 113_645, span(768, 120_000)])
    dim = rng.choice([64 * span(2, 64), 8 * span(8, 512), span(64, 4096)])
    dim += dim == 3072
    if op == "plan":
        n = span(1, 16_384)
        c = {"op": op, "requests": n, "tokens": rng.choice([0, 1]) * (n + span(16, 1_500_000)),
             "cached": rng.choice([0, span(1, 30_000)]), "block": rng.choice([1, 8, 16, 16, 32, 64, 100, 128, 256]),
             "free": rng.choice([1.0, 1.0, 0.7]), "pad": rng.randrange(0, 300)}
        c["cached"] = min(c["cached"], (16_000_000 * c["block"]) // n)
        shrink = ("tokens", "requests")
    elif op == "embed":
        w = rng.choice(["f32", "f16", "bf16", "bf16"])
        c = {"op": op, "tokens": span(1, 131_072), "rows": rows, "dim": dim, "weight": w,
             "out": rng.choice([w, "bf16"]), "scale": rng.choice([1.0, 8.0, 45.25])}
        shrink = ("tokens",)
    elif op == "grad":
        g = rng.choice(["f32", "f16", "bf16", "bf16"])
        c = {"op": op, "tokens": span(1, 131_072), "rows": rows, "dim": dim, "grad": g,
             "weight": rng.choice([g, "f32"]), "scale": rng.choice([1.0, 8.0, 45.25])}
        shrink = ("tokens", "dim", "rows")
    else:
        t = rng.choice(["f32", "f16", "bf16", "bf16"])
        c = {"op": op, "requests": span(1, 384), "vocab": rows, "prompt": rng.choice([0, span(10, 8000)]),
             "output": rng.choice([0, span(1, 2000)]), "bias": rng.choice([0, span(1, 300)]),
             "masks": rng.choice([0.0, 0.3, 1.0]), "logits": t, "out": rng.choice([t, "f32"])}
        shrink = ("requests",)
    for key in shrink:
        while work(c)["bytes"] > MOST[op] and c[key] > 1:
            c[key] = c[key] * 7 // 8
    if op in ("embed", "grad"):
        c["dim"] += c["dim"] == 3072
    return c


# ------------------------------------------------------------------ inputs --

def _frequencies(rows):
    """How often the id of each rank is met: a Zipf law as in the text workloads."""
    p = np.arange(1, rows + 1, dtype=np.float64) ** -1.1
    return p / p.sum()


def _ids(gen, n, rows):
    """n ids, frequent and rare ones mixed over the whole table."""
    cum = torch.from_numpy(np.cumsum(_frequencies(rows))).cuda()
    rank = torch.searchsorted(cum, torch.rand(n, generator=gen, device="cuda", dtype=torch.float64))
    step = 7919 if rows % 7919 else 7907
    return (rank.clamp_(max=rows - 1) * step % rows).to(torch.int32)


def _cuts(gen, n, total):
    """Offsets of n ragged parts of `total`, empty ones among them."""
    cuts = torch.randint(0, total + 1, (n - 1,), generator=gen, device="cuda").sort().values
    ends = torch.tensor([0, total], device="cuda")
    return torch.cat([ends[:1], cuts, ends[1:]])


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
    op = case["op"]

    def normal(*shape, dtype="f32", by=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * by).to(TYPES[dtype])

    if op == "plan":
        n, block = case["requests"], case["block"]
        # prompts of very different lengths, up to eight times the mean; what they leave of the tokens is padding
        longest = min(case["tokens"], 8 * case["tokens"] // n + 1) if case["tokens"] else 1
        s["offsets"] = None
        if case["tokens"]:
            share = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64) ** 4
            lens = (share / share.sum() * case["tokens"]).long().clamp(max=longest)
            s["offsets"] = torch.cat([torch.zeros_like(lens[:1]), lens.cumsum(0)])
        s["cached_lens"] = torch.randint(0, case["cached"] + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
        new = s["offsets"].diff() if case["tokens"] else torch.ones(n, dtype=torch.int64, device="cuda")
        held = (s["cached_lens"].long() + block - 1) // block
        want = (s["cached_lens"].long() + new + block - 1) // block
        width = (case["cached"] + longest + block - 1) // block
        need = int((want - held).sum())
        blocks = torch.randperm(n * width + need + 8, generator=gen, device="cuda").to(torch.int32)
        table = blocks[:n * width].reshape(n, width).clone()
        table[torch.arange(width, device="cuda") >= held[:, None]] = -1
        s["table"] = table
        s["free_blocks"] = blocks[n * width:][:int(need * case["free"]) + 3].clone()
        s["head"] = torch.full((1,), 3, dtype=torch.int64, device="cuda")
        s["slots"] = (case["tokens"] or n) + case["pad"]
    elif op == "embed":
        s["ids"] = _ids(gen, case["tokens"], case["rows"])
        s["table"] = normal(case["rows"], case["dim"], dtype=case["weight"], by=0.02)
    elif op == "grad":
        s["ids"] = _ids(gen, case["tokens"], case["rows"])
        s["upstream"] = normal(case["tokens"], case["dim"], dtype=case["grad"], by=0.1)
    else:
        n, vocab = case["requests"], case["vocab"]
        s["scores"] = normal(n, vocab, dtype=case["logits"], by=4.0)
        s["prompt_ids"], s["prompt_offsets"] = None, None
        if case["prompt"]:
            s["prompt_offsets"] = _cuts(gen, n, n * case["prompt"])
            s["prompt_ids"] = _ids(gen, n * case["prompt"], vocab)
        s["output_ids"], s["output_lens"] = None, None
        if case["output"]:
            s["output_ids"] = _ids(gen, n * (case["output"] + 5), vocab).reshape(n, -1)
            s["output_lens"] = torch.randint(0, case["output"] + 1, (n,), generator=gen, device="cuda",
                                             dtype=torch.int32)
        for name, lo, hi in (("repetition", 1.0, 1.5), ("frequency", 0.0, 0.6), ("presence", -0.2, 0.8)):
            s[name] = torch.rand(n, generator=gen, device="cuda") * (hi - lo) + lo
        s["bias_ids"] = None
        if case["bias"]:
            s["bias_offsets"] = _cuts(gen, n, n * case["bias"])
            s["bias_ids"] = _ids(gen, n * case["bias"], vocab)
            s["bias_values"] = normal(n * case["bias"], by=5.0)
        s["mask"], s["mask_rows"] = None, None
        masks = int(math.ceil(n * case["masks"]))
        if masks:
            # a grammar's mask: whole words of 32 ids are open or shut, or open here and there
            words = (vocab + 31) // 32
            bits = torch.randint(-2 ** 31, 2 ** 31, (masks, words), generator=gen, device="cuda")
            kind = torch.rand(masks, words, generator=gen, device="cuda")
            bits[kind < 0.5] = 0
            bits[kind > 0.8] = -1
            s["mask"] = bits.to(torch.int32)
            rows = torch.full((n,), -1, dtype=torch.int32, device="cuda")
            rows[torch.randperm(n, generator=gen, device="cuda")[:masks]] = torch.arange(masks, dtype=torch.int32,
                                                                                         device="cuda")
            s["mask_rows"] = rows
    return s


# -------------------------------------------------------------------- pass --

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_plan(s):
    seq_lens, slots, positions, info = s["tok"].plan_blocks(s["offsets"], s["cached_lens"], s["table"],
                                                            s["free_blocks"], s["block"], n_slots=s["slots"],
                                                            head=s["head"])
    return {"table": s["table"], "seq_lens": seq_lens, "slots": slots, "positions": positions, "info": info}


def _own_embed(s):
    return s["tok"].embed(s["ids"], s["table"], scale=s["scale"], dtype=TYPES[s["out"]])


def _own_grad(s):
    return s["tok"].embed_grad(s["ids"], s["upstream"], s["rows"], scale=s["scale"], dtype=TYPES[s["weight"]])


def _own_logits(s):
    return s["tok"].adjust_logits(
        s["scores"],
        prompt=(s["prompt_ids"], s["prompt_offsets"]) if s["prompt_ids"] is not None else None,
        output=(s["output_ids"], s["output_lens"]) if s["output_ids"] is not None else None,
        repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
        bias=(s["bias_ids"], s["bias_values"], s["bias_offsets"]) if s["bias_ids"] is not None else None,
        mask=s["mask"], mask_rows=s["mask_rows"], dtype=TYPES[s["out"]])


_own = {"plan": _own_plan, "embed": _own_embed, "grad": _own_grad, "logits": _own_logits}


def _owner(offsets, n, total):
    """Which part each of `total` places belongs to."""
    marks = torch.zeros(total + 1, dtype=torch.int64, device="cuda")
    marks.index_add_(0, offsets[1:n], torch.ones(n - 1, dtype=torch.int64, device="cuda"))
    return marks[:total].cumsum(0)


def _plain_plan(s):
    n, block, table, free = s["requests"], s["block"], s["table"], s["free_blocks"]
    cached, head, slots = s["cached_lens"].long(), s["head"], s["slots"]
    offsets = s["offsets"] if s["offsets"] is not None else torch.arange(n + 1, device="cuda")
    new = offsets[1:] - offsets[:-1]
    held = (cached + block - 1) // block
    gets = (cached + new + block - 1) // block - held
    upto = gets.cumsum(0)
    room = free.numel() - head
    served = (gets == 0) | (upto <= room)
    # the blocks that the requests get, in place
    k = torch.arange(table.shape[1], device="cuda")[None, :] - held[:, None]
    fresh = served[:, None] & (k >= 0) & (k < gets[:, None])
    at = (head + (upto - gets)[:, None] + k).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[at], table))
    seq_lens = torch.where(served, cached + new, cached).to(torch.int32)
    t = torch.arange(slots, device="cuda")
    real = t < offsets[-1]
    i = _owner(offsets, n, slots)
    position = torch.where(real, cached[i] + t - offsets[i], 0)
    slot = table[i, position // block].long() * block + position % block
    slot = torch.where(real & served[i], slot, -1)
    taken = torch.where(upto <= room, upto, 0).max()
    info = torch.stack([head[0] + taken, (upto[-1] - room[0]).clamp(min=0)])
    return {"table": table, "seq_lens": seq_lens, "slots": slot, "positions": position.to(torch.int32), "info": info}


def _plain_embed(s):
    return (s["table"][s["ids"].long()].float() * s["scale"]).to(TYPES[s["out"]])


def _plain_grad(s):
    total = torch.zeros(s["rows"], s["dim"], dtype=torch.float32, device="cuda")
    total.index_add_(0, s["ids"].long(), s["upstream"].float())
    return (total * s["scale"]).to(TYPES[s["weight"]])


def _plain_logits(s):
    n, vocab = s["requests"], s["vocab"]
    x = s["scores"].float()
    times = torch.zeros(n * vocab, device="cuda")
    if s["output_ids"] is not None:
        width = s["output_ids"].shape[1]
        there = torch.arange(width, device="cuda")[None, :] < s["output_lens"][:, None]
        flat = torch.arange(n, device="cuda")[:, None] * vocab + s["output_ids"].long()
        times.index_add_(0, flat.reshape(-1), there.reshape(-1).float())
    seen = times > 0
    if s["prompt_ids"] is not None:
        total = s["prompt_ids"].numel()
        seen[_owner(s["prompt_offsets"], n, total) * vocab + s["prompt_ids"].long()] = True
    times, seen = times.reshape(n, vocab), seen.reshape(n, vocab)
    by = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / by, x * by), x)
    x = x - s["frequency"][:, None] * times - s["presence"][:, None] * (times > 0).float()
    if s["bias_ids"] is not None:
        total = s["bias_ids"].numel()
        add = torch.zeros(n * vocab, device="cuda")
        add.index_add_(0, _owner(s["bias_offsets"], n, total) * vocab + s["bias_ids"].long(), s["bias_values"])
        x = x + add.reshape(n, vocab)
    if s["mask"] is not None:
        v = torch.arange(vocab, device="cuda")
        rows = s["mask_rows"].long()
        bits = s["mask"][:, v // 32] >> (v % 32).to(torch.int32) & 1
        shut = (bits[rows.clamp(min=0)] == 0) & (rows >= 0)[:, None]
        x = torch.where(shut, -math.inf, x)
    return x.to(TYPES[s["out"]])


_plain = {"plan": _plain_plan, "embed": _plain_embed, "grad": _plain_grad, "logits": _plain_logits}


# ----------------------------------------------------------- what it needs --

def work(case):
    op = case["op"]
    if op == "plan":
        n, block = case["requests"], case["block"]
        new = case["tokens"] or n
        blocks = new / block
        return {"bytes": (8 * (n + 1) if case["tokens"] else 0) + 4 * n + 4 * n + 8 * blocks + 4 * n
                + 12 * ((case["tokens"] or n) + case["pad"]) + 24, "flops": 0}
    if op == "embed":
        met = float((1 - (1 - _frequencies(case["rows"])) ** case["tokens"]).sum())
        return {"bytes": 4 * case["tokens"] + met * case["dim"] * SIZE[case["weight"]]
                + case["tokens"] * case["dim"] * SIZE[case["out"]], "flops": case["tokens"] * case["dim"]}
    if op == "grad":
        return {"bytes": 4 * case["tokens"] + case["tokens"] * case["dim"] * SIZE[case["grad"]]
                + case["rows"] * case["dim"] * SIZE[case["weight"]], "flops": case["tokens"] * case["dim"]}
    n, vocab = case["requests"], case["vocab"]
    words = (vocab + 31) // 32
    return {"bytes": n * vocab * (SIZE[case["logits"]] + SIZE[case["out"]])
            + 4 * words * math.ceil(n * case["masks"]) + n * (4 * case["prompt"] + 2 * case["output"] + 12)
            + 8 * n * case["bias"] + 8 * n, "flops": 2 * n * vocab}


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "embed":
        ids, scale = s["ids"].cpu().numpy(), float(np.float32(case["scale"]))
        table = s["table"].float().cpu().numpy()
        return torch.from_numpy(np.take(table, ids, axis=0).astype(np.float64) * scale)
    if op == "grad":
        # sorted by id, the sums are differences of running sums, taken a few columns at a time
        ids, order = s["ids"].long().sort(stable=True)
        first = torch.searchsorted(ids, torch.arange(case["rows"] + 1, device="cuda"))
        out = torch.empty(case["rows"], case["dim"], dtype=torch.float64, device="cuda")
        for c in range(0, case["dim"], 256):
            run_ = s["upstream"][:, c:c + 256].double()[order].cumsum(0)
            run_ = torch.cat([torch.zeros_like(run_[:1]), run_])
            out[:, c:c + 256] = run_[first[1:]] - run_[first[:-1]]
        return out * case["scale"]
    # logits: a request at a time on the host
    vocab = case["vocab"]
    host = {k: v.cpu().numpy() for k, v in s.items() if isinstance(v, torch.Tensor) and k != "scores"}
    out = np.empty((case["requests"], vocab))
    for b in range(case["requests"]):
        x = s["scores"][b].double().cpu().numpy()
        said = host["output_ids"][b, :host["output_lens"][b]] if case["output"] else np.zeros(0, np.int32)
        times = np.bincount(said, minlength=vocab)
        seen = times > 0
        if case["prompt"]:
            lo, hi = host["prompt_offsets"][b:b + 2]
            seen[host["prompt_ids"][lo:hi]] = True
        by = float(host["repetition"][b])
        x[seen] = np.where(x[seen] > 0, x[seen] / by, x[seen] * by)
        x -= float(host["frequency"][b]) * times + float(host["presence"][b]) * (times > 0)
        if case["bias"]:
            lo, hi = host["bias_offsets"][b:b + 2]
            np.add.at(x, host["bias_ids"][lo:hi], host["bias_values"][lo:hi].astype(np.float64))
        row = host["mask_rows"][b] if case["masks"] else -1
        if row >= 0:
            x[np.unpackbits(host["mask"][row].view(np.uint8), bitorder="little")[:vocab] == 0] = -np.inf
        out[b] = x
    return torch.from_numpy(out)
