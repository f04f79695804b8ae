"""Attention over a cache in 4 bits in 64 bits, with a bound that the kernels'
roundings keep to and that a wrong scale, mask or weight does not."""
from __future__ import annotations

import numpy as np

from tests import paged_util as pu
from tests.ops_util import assert_close

U = 2.0 ** -24   # half a step of float32, relative
H = 2.0 ** -11   # of a half
SURE = 6.0       # see below


def request_rows(cache, table_row, length, h, block, dim):
    """float64 ((keys, steps, bases, codes), (the same of values)) of a request's first tokens in head h."""
    out = []
    blocks = -(-length // block)
    for which in (0, 1):
        codes, pairs = [np.zeros((0, pu.groups(dim) * 32), np.uint8)], [np.zeros((0, pu.groups(dim)), np.uint32)]
        for b in table_row[:blocks]:
            c, p = pu.unpack(cache[b, which, h], block, dim)
            codes.append(c), pairs.append(p)
        code, pair = np.concatenate(codes)[:length], np.concatenate(pairs)[:length]
        step, base = pu.bf16_value(pair & 0xFFFF).astype(np.float64), pu.bf16_value(pair >> 16).astype(np.float64)
        code = code[:, :dim].astype(np.float64)
        s, b = np.repeat(step, 32, 1)[:, :dim], np.repeat(base, 32, 1)[:, :dim]
        out.append((b + s * code, s, b, code))
    return out


def spread(x, dim):
    """[.., dim] to [.., groups, 32], zeros behind."""
    g = pu.groups(dim)
    return np.pad(x, [(0, 0)] * (x.ndim - 1) + [(0, g * 32 - dim)]).reshape(*x.shape[:-1], g, 32)


def attention(q, cache, table, lens, block, offsets=None, scale=None, parts=1):
    """(out, bound) of attend for float64 queries [tokens, rows, dim] of a type that `parts` halves hold (1 of 16
    bits, 2 of 32); NaN where no request has the token.

    out_i = sum_t p_t v_ti. An error d_t of a score changes it by sum_t p_t d_t (v_ti - out_i), a relative error e_t of
    a weight (or of the value under it) by sum_t p_t e_t v_ti. Errors that may have one sign for all tokens are added
    up. Roundings to a half (of weights, and in long runs of keys and values) fall either way, independently from
    token to token: with |e_t| <= c_t, Hoeffding's inequality holds their sum below SURE * sqrt(sum c_t^2) but for 2
    e^-18 of all elements; real roundings have less than a third of that variance, and every input here is fixed.

    Scores. 32-bit steps: products with scale and log2 e, the subtraction of the maximum, the exponential (4 U):
    8 U (|s_t| + max |s|). Bases: sums of a group's queries, three parts of bfloat16, 48 products cut off 23 bits below
    the largest: 128 U sum |B x|. Codes, one part: a query scaled to 2^14..2^15 times a code is cut at 2^-24 of the
    code's unit times 2, so an element loses up to 2 units where its own last bit is below the unit (an fp16 or bf16
    one cannot below 2^-4 or 2^-7 of the largest), and two more for the sums beyond 2^24. Two parts: 34 products of up
    to 16 |x| S cut off 23 bits below the largest, and |x| to 2 U of itself and 2^-39 of the largest. Long runs: keys
    to H of themselves either way, dim + 16 products cut off 23 bits below the largest, and queries scaled to
    2^6..2^7 that a half may not hold, off by 2^-25.

    Weights, one part: H for the weight, and H again for its product with a step, or for the middle of a group's
    values; sizes are those of S n and S (n - 8), and of B and B + 8 S. Long runs: H for the weight and H for the
    value. Two parts: 2^-20 for everything. Cut-off sums: 68 U a step of 32 tokens, and tokens / 8 + 64 roundings of
    2 U. What lies below a half's smallest numbers: values are halves where a share's sizes are within 2^12 of each
    other (2^8 of them the largest), and its largest weight is 2^11, so that a token loses 2^-23 of the largest p size
    (at most the root of the sum of their squares); in long runs steps lose 2^-21 where the largest of the first
    tokens is 2^6 and what is below 2^-9 is done otherwise, and weights 2^-31 of the largest."""
    tokens, rows, dim = q.shape
    heads = cache.shape[2]
    group = rows // heads
    scale = dim ** -0.5 if scale is None else scale
    out, bound = np.full(q.shape, np.nan), np.zeros(q.shape)
    n = len(lens)
    many = offsets is not None and parts == 1 and tokens * rows >= 8192  # long runs are those of 64 columns and more
    offsets = np.arange(n + 1) if offsets is None else np.asarray(offsets)
    for r in range(n):
        first, m, length = int(offsets[r]), int(offsets[r + 1] - offsets[r]), int(lens[r])
        if m == 0:
            continue
        long = many and m * group >= 64
        for h in range(heads):
            (k, ks, kb, _), (v, vs, vb, vn) = request_rows(cache, table[r], length, h, block, dim)
            x = q[first:first + m, h * group:(h + 1) * group].reshape(m * group, dim)
            seen = np.clip(length - m + np.repeat(np.arange(m), group) + 1, 0, length)
            see = np.arange(length)[None, :] < seen[:, None]
            if length == 0:
                out[first:first + m, h * group:(h + 1) * group] = 0
                continue
            s = scale * (x @ k.T)
            top = np.where(see, s, -np.inf).max(1, keepdims=True)
            top[np.isinf(top)] = 0
            w = np.where(see, np.exp(np.minimum(s - top, 0)), 0)
            total = w.sum(1, keepdims=True)
            p = w / np.maximum(total, 1)  # a weight of one is among them, or all are zero
            y = p @ v
            # scores
            ax, biggest = np.abs(x), np.abs(x).max(1, keepdims=True)
            lin = 8 * U * (np.abs(s) + np.abs(np.where(see, s, 0)).max(1, keepdims=True))
            lin += 128 * U * abs(scale) * (ax @ np.abs(kb).T)
            steps = np.abs(spread(ks, dim)[..., 0])
            exponent = np.frexp(np.where(biggest > 0, biggest, 1))[1] - 1 - 14  # 2^exponent: the unit of a scaled code
            if parts == 1:
                unit = np.ldexp(1.0, exponent)
                fine = spread((ax > 0) & (np.remainder(ax / unit, 1) != 0), dim).sum(-1)
                lin += abs(scale) * 2 * unit * ((fine + 2.0 * spread(ax > 0, dim).any(-1)) @ steps.T)
                small = 2.0 ** (8 if long else 0) * unit
                lin += abs(scale) * 2.0 ** -25 * small * ((np.remainder(ax / (small * 2.0 ** -24), 1) != 0) @ np.abs(k).T)
            else:
                lin += abs(scale) * 34 * 2 * U * 16 * (spread(ax, dim).max(-1) @ steps.T)
                lin += abs(scale) * (2 * U * ax + 2.0 ** -39 * biggest * (ax > 0)) @ np.abs(k).T
            size = np.abs(vs) * np.maximum(vn, np.abs(vn - 8)) + np.maximum(np.abs(vb), np.abs(vb + 8 * vs))
            either = np.zeros_like(s)
            if long:
                either = abs(scale) * H * np.sqrt((x ** 2) @ (k ** 2).T)
                largest = spread(ax, dim).max(-1)[:, None] * spread(np.abs(k), dim).max(-1)[None]
                lin += abs(scale) * (dim + 16) * 2 * U * largest.max(-1)
            grow = np.exp(2 * np.where(p > 0, lin + SURE * either, 0).max(1, keepdims=True))
            off = ((p * lin) @ np.abs(v) + (p * lin).sum(1, keepdims=True) * np.abs(y)) * grow
            p2 = (p * either) ** 2
            off += SURE * np.sqrt(np.maximum(p2 @ v ** 2 - 2 * y * (p2 @ v) + p2.sum(1, keepdims=True) * y ** 2, 0)) * grow
            # weights
            if parts == 1:
                off += SURE * H * np.sqrt(2 * (p ** 2) @ size ** 2)
            off += ((2.0 ** -20 if parts == 2 else 0) + 68 * U + (length / 8 + 64) * 2 * U) * (p @ size)
            off += length * 2.0 ** -23 * np.sqrt((p ** 2) @ size ** 2)
            if long:
                off += p @ np.minimum(2.0 ** -27 * size.max(), 2.0 ** -12 * size)
                off += 2.0 ** -31 * (see @ size) / np.maximum(total, 1)
            y[seen == 0], off[seen == 0] = 0, 0
            out[first:first + m, h * group:(h + 1) * group] = y.reshape(m, group, dim)
            bound[first:first + m, h * group:(h + 1) * group] = off.reshape(m, group, dim)
    return out, bound


def scale_pairs(b, which, exponent, r=None, t=None, group=None, set_to=None):
    """Multiplies steps and bases of keys (0) or values (1) by 2^exponent, or sets their words: of all tokens or of
    token t of request r, in all groups or in one."""
    g = pu.groups(b.dim)
    at = b.block * g * 16
    words = b.cache[:, which, :, at:at + b.block * g * 4].copy().view("<u4").reshape(
        len(b.cache), -1, b.block, g)
    blocks = slice(None) if r is None else b.table[r, t // b.block]
    rows = slice(None) if r is None else t % b.block
    columns = slice(None) if group is None else group
    old = words[blocks, :, rows, columns]
    if set_to is not None:
        new = np.full_like(old, set_to)
    else:
        f = np.float32(2.0) ** exponent
        new = pu.bf16_bits(pu.bf16_value(old & 0xFFFF) * f) | pu.bf16_bits(pu.bf16_value(old >> 16) * f) << np.uint32(16)
    words[blocks, :, rows, columns] = new
    b.cache[:, which, :, at:at + b.block * g * 4] = words.reshape(len(b.cache), words.shape[1], -1).view(np.uint8)


def check(tok, b, label="", **k):
    """attend of a Batch (test_gpu_attend.py) within its bound."""
    import torch
    got = b.run(tok, **k)
    name = str(b.q.dtype).replace("torch.", "")
    want, bound = attention(b.q.double().numpy(), b.cache, b.table, b.lens, b.block, b.offsets, k.get("scale"),
                            2 if name == "float32" else 1)
    none = np.isnan(want).all((1, 2))  # tokens of no request
    assert not bool(got[torch.from_numpy(none).cuda()].any())
    assert_close(got[torch.from_numpy(~none).cuda()], torch.from_numpy(want[~none]), torch.from_numpy(bound[~none]), label)
    return got
