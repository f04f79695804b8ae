"""Plain forms of the operators on a paged cache in 4 bits, in numpy on the
host: the cache's layout and rounding bit by bit, rotations and attention in 64
bits, with bounds of what 32-bit kernels may be off by."""
from __future__ import annotations

import math

import numpy as np

GROUP = 32
U = 2.0 ** -24  # half a step of float32


def groups(dim):
    g = -(-dim // GROUP)
    return g if g <= 4 or g % 2 == 0 else g + 1


def page_bytes(block, dim):
    return -(-(block * groups(dim) * 20) // 16) * 16


def code_place(e, dim):
    """Where element e's code lies in a row, counted in codes."""
    j, i = divmod(e, GROUP)
    g = groups(dim)
    if g % 2 and j == g - 1:
        return e
    return (j // 2) * 64 + (i // 8) * 16 + (j % 2) * 8 + i % 8


def bf16_bits(x):
    """The nearest bfloat16 of float32, ties to even, as its bits."""
    b = np.atleast_1d(np.asarray(x, np.float32)).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> np.uint64(16)) & np.uint64(1))) >> np.uint64(16)
    return b.astype(np.uint32).reshape(np.shape(x))


def bf16_value(bits):
    return (np.asarray(bits, np.uint32) << np.uint32(16)).view(np.float32)


def quantise(row, dim):
    """(codes uint8[groups * 32], pairs uint32[groups]) of a float32 row."""
    f = np.float32
    codes, pairs = np.zeros(groups(dim) * GROUP, np.uint8), np.zeros(groups(dim), np.uint32)
    for j in range(groups(dim)):
        x = np.asarray(row[j * GROUP:min(dim, (j + 1) * GROUP)], f)
        if x.size == 0:
            continue
        if not np.all(np.abs(x) <= f(3.3895314e38)):
            pairs[j] = 0x7FC00000
            continue
        base_bits = bf16_bits(x.min())
        half = f(0.5) * bf16_value(base_bits)
        step_bits = bf16_bits(max((f(0.5) * x.max() - half) * (f(1) / f(7.5)), f(0)))
        step = bf16_value(step_bits)
        if step < 2.0 ** -100:
            step_bits, step = np.uint32(0), f(0)
        by = f(1) / (f(0.5) * step) if step > 0 else f(0)
        codes[j * GROUP:j * GROUP + x.size] = np.clip(np.rint((f(0.5) * x - half) * by), 0, 15)
        pairs[j] = step_bits | base_bits << np.uint32(16)
    return codes, pairs


def value(codes, pairs, dim):
    """float32 that a row stands for (its one rounding is the sum's)."""
    step, base = bf16_value(pairs & 0xFFFF), bf16_value(pairs >> 16)
    with np.errstate(invalid="ignore"):
        v = np.repeat(base, GROUP) + np.repeat(step, GROUP) * codes.astype(np.float32)
    return v[:dim]


def put_row(page, block, dim, place, codes, pairs):
    """Writes a row into a page (uint8 array)."""
    g = groups(dim)
    packed = np.zeros(g * 16, np.uint8)
    for e in range(g * GROUP):
        at = code_place(e, dim)
        packed[at // 2] |= codes[e] << (4 * (at % 2))
    page[place * g * 16:(place + 1) * g * 16] = packed
    at = block * g * 16 + place * g * 4
    page[at:at + g * 4] = np.ascontiguousarray(pairs, dtype="<u4").view(np.uint8)


def unpack(page, block, dim):
    """(codes uint8[block, groups * 32], pairs uint32[block, groups]) of a page."""
    g = groups(dim)
    packed = page[:block * g * 16].reshape(block, g * 16)
    place = np.array([code_place(e, dim) for e in range(g * GROUP)])
    codes = packed[:, place // 2] >> (4 * (place % 2)).astype(np.uint8) & 15
    pairs = np.ascontiguousarray(page[block * g * 16:block * g * 20]).view("<u4").reshape(block, g)
    return codes, pairs


def random_cache(rng, blocks, heads, block, dim):
    """A cache whose rows stand for about normal values, padding of any content."""
    cache = rng.integers(0, 256, (blocks, 2, heads, page_bytes(block, dim)), dtype=np.uint8)
    g = groups(dim)
    step = rng.uniform(0.1, 0.3, (blocks, 2, heads, block * g)).astype(np.float32)
    base = (-8 * step + 0.3 * rng.standard_normal(step.shape)).astype(np.float32)
    pairs = bf16_bits(step) | bf16_bits(base) << np.uint32(16)
    cache[..., block * g * 16:block * g * 20] = np.ascontiguousarray(pairs, dtype="<u4").view(np.uint8)
    return cache


def attention(q, cache, table, lens, block, offsets=None, scale=None, parts=1):
    """(out, bound) in 64 bits: what attend gives for float64 queries [tokens,
    rows, dim], and what its sums may be off by. NaN where no request has the
    token. parts: halves that a weight or a query is cut into (1 for 16-bit
    queries, 2 for 32-bit ones).

    The bound, with u = 2^-24 and the tensor cores' sums taken to lose up to 2 u
    of what they hold at each of their additions. A score's sums have at most
    dim + 3 groups additions of terms below |q_i| (48 step + |base|), and its
    products with scale and log2 e two roundings of |s|. With one part, keys are
    halves, off by 2^-12 of themselves, or codes as subnormal halves, whose
    products lose what lies 24 bits below their exponent's 2^-14: of queries
    scaled to 2^14 at most 2^-13 of the largest, times the step. e^x is off by 2 u
    and by the error of its argument, a score's and the maximum's. A weight is
    rounded twice, or once and its value once, to 2^-(12 parts) each. The sum over
    tokens is one of at most tokens + 64 additions of terms below p (48 step +
    |base|), the joining of parts among them."""
    tokens, rows, dim = q.shape
    heads = cache.shape[2]
    group = rows // heads
    scale = dim ** -0.5 if scale is None else scale
    out, bound = np.full(q.shape, np.nan), np.zeros(q.shape)
    n = len(lens)
    offsets = np.arange(n + 1) if offsets is None else np.asarray(offsets)
    g = groups(dim)
    for r in range(n):
        first, m = int(offsets[r]), int(offsets[r + 1] - offsets[r])
        length = int(lens[r])
        if m == 0:
            continue
        for h in range(heads):
            kv, size, steps = [], [], []
            for which in (0, 1):
                rows_c, rows_p = [], []
                for b in range(-(-length // block)):
                    c, p = unpack(cache[table[r, b], which, h], block, dim)
                    rows_c.append(c)
                    rows_p.append(p)
                c = np.concatenate(rows_c)[:length] if rows_c else np.zeros((0, g * GROUP), np.uint8)
                p = np.concatenate(rows_p)[:length] if rows_p else np.zeros((0, g), np.uint32)
                step, base = bf16_value(p & 0xFFFF).astype(np.float64), bf16_value(p >> 16).astype(np.float64)
                with np.errstate(invalid="ignore"):
                    kv.append((np.repeat(base, GROUP, 1) + np.repeat(step, GROUP, 1) * c)[:, :dim])
                steps.append(step)
                size.append(np.repeat(48 * step + np.abs(base), GROUP, 1)[:, :dim])
            for i in range(m):
                seen = min(max(length - m + i + 1, 0), length)
                for k in range(group):
                    at = (first + i, h * group + k)
                    if seen == 0:
                        out[at] = 0
                        continue
                    x = q[at]
                    with np.errstate(invalid="ignore"):
                        s = scale * (kv[0][:seen] @ x)
                        off = abs(scale) * (size[0][:seen] @ np.abs(x)) * (dim + 3 * g) * 2 * U + 4 * U * np.abs(s)
                        if parts == 1:
                            off += abs(scale) * (size[0][:seen] @ np.abs(x)) * 2.0 ** -12
                            off += abs(scale) * np.abs(x).max() * 2.0 ** -13 * 34 * steps[0][:seen].sum(1)
                        w = np.exp(s - s.max())
                        w /= w.sum()
                        out[at] = w @ kv[1][:seen]
                        rel = 2 * off.max() + 4 * U * (s.max() - s.min() + 1) + 4 * U
                        rel += 2.0 ** -(12 * parts - 1) + (seen + 64) * 2 * U
                        bound[at] = np.expm1(rel) * (w @ size[1][:seen])
    return out, bound


def turned(x, positions, frequencies, interleaved, scale, inverse=False):
    """(y, bound) in 64 bits of float64 x [tokens, heads, dim]. The bound in half
    steps u of float32: the angle, rounded to 2^-24 of at most a half turn, pi u;
    its sine and cosine 2, the product with scale 1, products and sum 2."""
    pairs = len(frequencies)
    at = np.arange(pairs)
    a, b = (2 * at, 2 * at + 1) if interleaved else (at, pairs + at)
    angle = np.asarray(positions, np.float64)[:, None] * np.asarray(frequencies, np.float64)
    c, s = np.cos(angle)[:, None] * scale, np.sin(angle)[:, None] * scale * (-1 if inverse else 1)
    y, bound = x.copy(), np.zeros(x.shape)
    x1, x2 = x[..., a], x[..., b]
    y[..., a], y[..., b] = x1 * c - x2 * s, x1 * s + x2 * c
    bound[..., a] = bound[..., b] = (np.abs(x1) + np.abs(x2)) * abs(scale) * (math.pi + 5) * U
    return y, bound
