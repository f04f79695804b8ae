"""The step of a group is a quotient rounded to 32 bits and then to bfloat16:
groups whose quotient is a bfloat16 tie, which a product with 1 / 7.5 misses."""
import numpy as np
import pytest

from tests import paged_util as pu
from tests.ops_util import byte_tokenizer, load


def pairs_of(low, high):
    """(step, base) words of groups from `low` to `high`, float32, as the header states them."""
    f = np.float32
    base_bits = pu.bf16_bits(low)
    half = f(0.5) * pu.bf16_value(base_bits)
    step_bits = pu.bf16_bits(np.maximum((f(0.5) * high - half) / f(7.5), f(0)))
    step_bits[pu.bf16_value(step_bits) < 2.0 ** -100] = 0
    return step_bits | base_bits << np.uint32(16)


def ties(dtype, n):
    """n pairs (low, high) of float16 or float32 ends that a product with the rounded 1 / 7.5 gives another step."""
    rng = np.random.default_rng(7)
    found = []
    while sum(map(len, found)) < n:
        ends = np.sort(rng.normal(0, 0.7, (1 << 20, 2)).astype(dtype).astype(np.float32), 1)
        f = np.float32
        half = f(0.5) * ends[:, 1] - f(0.5) * pu.bf16_value(pu.bf16_bits(ends[:, 0]))
        other = pu.bf16_bits(half / f(7.5)) != pu.bf16_bits(half * (f(1) / f(7.5)))
        found.append(ends[other & (half > 0)])
    return np.concatenate(found)[:n]


def test_quotients_next_to_exact_ties_round_to_even():
    """Against exact arithmetic: where the quotient is a tie, the step is the even neighbour."""
    from fractions import Fraction
    exact = 0
    for low, high in ties(np.float16, 50):
        step = Fraction(float(pu.bf16_value(pairs_of(np.float32([low]), np.float32([high])) & 0xFFFF)[0]))
        base = Fraction(float(pu.bf16_value(pu.bf16_bits(np.float32([low])))[0]))
        want = (Fraction(float(high)) - base) / 15
        ulp = Fraction(2) ** (np.frexp(float(step))[1] - 8)
        assert abs(step - want) <= ulp / 2 * (1 + Fraction(1, 2 ** 14))
        if abs(step - want) == ulp / 2:
            exact += 1
            assert (step / ulp) % 2 == 0
    assert exact >= 10


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float16", "float32"])
@pytest.mark.parametrize("dim,block", [(64, 16), (96, 7)])
def test_steps_next_to_ties(dtype, dim, block):
    import torch
    tok = byte_tokenizer(load())
    groups = dim // 32
    ends = ties(np.dtype(dtype).type, 64 * groups if dtype == "float16" else 4 * groups)
    rng = np.random.default_rng(1)
    x = (ends[:, :1] + (ends[:, 1:] - ends[:, :1]) * rng.random((len(ends), 32))).astype(np.dtype(dtype).type)
    x[:, 3], x[:, 29] = ends[:, 0], ends[:, 1]
    x = np.clip(x.astype(np.float32), ends[:, :1], ends[:, 1:]).reshape(-1, 1, dim)
    n = len(x)
    d = torch.from_numpy(x).to(getattr(torch, dtype)).cuda()
    cache = tok.new_cache(n // block + 1, block, 1, dim)
    tok.write_cache(cache, torch.arange(n, device="cuda"), d, d, block)
    got = cache.cpu().numpy()
    want = pairs_of(ends[:, 0], ends[:, 1]).reshape(n, groups)
    for which in (0, 1):
        pairs = np.concatenate([pu.unpack(got[b, which, 0], block, dim)[1] for b in range(len(got))])[:n]
        assert np.array_equal(pairs, want)
    # codes are to the nearest of the steps, so that what is read is off by half a step and the largest's rounding
    k, _ = tok.read_cache(cache, torch.arange(n, device="cuda"), dim, block)
    step = np.repeat(pu.bf16_value(want & 0xFFFF).reshape(n, 1, groups), 32, 2)
    off = np.abs(k.cpu().numpy().astype(np.float64) - x)
    over = np.maximum(0, x - (np.repeat(pu.bf16_value(want >> 16).reshape(n, 1, groups), 32, 2) + 15.0 * step))
    assert np.all(off <= np.maximum(step * 0.5001, over + 1e-6) + 2.0 ** -8 * np.abs(x))
    tok.close()
