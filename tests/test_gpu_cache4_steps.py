"""The step of a group is a product with 1 / 7.5 in 32 bits, as the header defines
it: groups where the quotient is next to a bfloat16 tie and would be rounded to the
other neighbour. Codes follow the step, so what is read back is as good."""
import numpy as np
import pytest

from tests import paged_util as pu
from tests.ops_util import byte_tokenizer, load

F = np.float32


def halves(ends):
    return F(0.5) * ends[:, 1] - F(0.5) * pu.bf16_value(pu.bf16_bits(ends[:, 0]))


def next_to_ties(dtype, n):
    """n pairs (smallest, largest) of float16 or float32 for which quotient and product give different steps."""
    rng = np.random.default_rng(7)
    found = []
    while sum(map(len, found)) < n:
        ends = np.sort(rng.normal(0, 0.7, (1 << 20, 2)).astype(dtype).astype(F), 1)
        half = halves(ends)
        found.append(ends[(pu.bf16_bits(half / F(7.5)) != pu.bf16_bits(half * (F(1) / F(7.5)))) & (half > 0)])
    return np.concatenate(found)[:n]


def groups_of(ends):
    """Groups of 32 elements with these ends."""
    rng = np.random.default_rng(1)
    x = np.clip((ends[:, :1] + (ends[:, 1:] - ends[:, :1]) * rng.random((len(ends), 32))).astype(F), ends[:, :1], ends[:, 1:])
    x[:, 3], x[:, 29] = ends[:, 0], ends[:, 1]
    return x


def test_either_neighbour_is_as_good():
    """The two steps are neighbours next to whose middle the quotient lies, so the largest element is as far off."""
    for dtype, n in ((np.float16, 200), (np.float32, 8)):
        ends = next_to_ties(dtype, n)
        half = halves(ends).astype(np.float64)
        steps = np.stack([pu.bf16_value(pu.bf16_bits(s)).astype(np.float64) for s in (F(half) / F(7.5), F(half) * (F(1) / F(7.5)))])
        gap = np.abs(steps[0] - steps[1])
        assert np.all(gap <= 2.0 ** -7 * steps.min(0)) and np.all(gap > 0)
        assert np.all(np.abs(half / 7.5 - steps.mean(0)) <= gap * 2.0 ** -14)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float16", "float32"])
@pytest.mark.parametrize("dim,block", [(64, 16), (96, 7)])
def test_steps_next_to_ties(dtype, dim, block):
    import torch
    tok = byte_tokenizer(load())
    x = groups_of(next_to_ties(np.dtype(dtype).type, dim // 32 * (64 if dtype == "float16" else 4)))
    d = torch.from_numpy(x.reshape(-1, 1, dim)).to(getattr(torch, dtype))
    n, rows = len(d), d.float().numpy()[:, 0]
    cache = tok.new_cache(n // block + 1, block, 1, dim)
    slots = torch.arange(n, device="cuda")
    tok.write_cache(cache, slots, d.cuda(), d.cuda(), block)
    got = cache.cpu().numpy()
    want = np.zeros_like(got)
    for t in range(n):
        for which in (0, 1):
            pu.put_row(want[t // block, which, 0], block, dim, t % block, *pu.quantise(rows[t], dim))
    assert np.array_equal(got, want)
    # half a step, or what the largest element is beyond the last of 15 steps
    k, _ = tok.read_cache(cache, slots, dim, block)
    off = np.abs(k.cpu().numpy()[:, 0].astype(np.float64) - rows).reshape(n, -1, 32)
    pairs = np.stack([pu.quantise(r, dim)[1] for r in rows])
    step, base = (pu.bf16_value(w).astype(np.float64)[..., None] for w in (pairs & 0xFFFF, pairs >> 16))
    beyond = np.maximum(rows.reshape(n, -1, 32) - (base + 15 * step), base - rows.reshape(n, -1, 32))
    assert np.all(off <= np.maximum(step * 0.5001, beyond) + 2.0 ** -20)
    tok.close()
