"""Attention over values of very different sizes: groups of a head's elements,
and tokens, up to 2^60 apart. What a column's sums hold of one must not depend on
how large another is."""
import numpy as np
import pytest

from tests import paged_util as pu
from tests.ops_util import byte_tokenizer, load
from tests.paged_close import check, scale_pairs
from tests.test_gpu_attend import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tok():
    t = byte_tokenizer(load())
    yield t
    t.close()


DTYPES = ["float32", "float16", "bfloat16"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 96, 128, 200, 256])
@pytest.mark.parametrize("new", [None, [1, 3, 5]])
def test_groups_of_values_apart(tok, dim, dtype, new):
    """Results of a group of channels 2^k smaller than another are as good as by themselves."""
    import torch
    for k in (5, 9, 12, 16, 20, 24, 40, 60):
        b = Batch([1, 170, 333], 2, 2, dim, 16, dtype, new=new, seed=dim + k)
        scale_pairs(b, 1, 20, group=0)  # fp16 results stay below their largest, 65504, and above their smallest
        scale_pairs(b, 1, 20 - k, group=1)
        if dtype == "float16":
            check(tok, b, k, dtype=torch.float32)
        else:
            check(tok, b, k)


def late_and_large(b, exponent, weight, group=None):
    """One token of each request, in its middle, has values 2^exponent larger and the score -weight, about."""
    import torch
    b.q = b.q.abs()
    mean = float(b.q.double().mean()) * b.dim * b.dim ** -0.5
    base = int(pu.bf16_bits(np.float32(-weight / mean)))
    for r, length in enumerate(b.lens):
        if length < 3:
            continue
        t = int(length) // 2
        scale_pairs(b, 0, 0, r, t, set_to=base << 16)
        scale_pairs(b, 1, exponent, r, t, group)
    assert b.q.dtype is not torch.float64


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [32, 72, 128, 256])
@pytest.mark.parametrize("new", [None, [1, 4, 40]])
def test_tokens_of_values_apart(tok, dim, dtype, new):
    """A token 2^k larger with a weight of e^-40 leaves the others what is theirs."""
    for k in (4, 8, 12, 20, 30, 45):
        for group in (None, 0):
            b = Batch([2, 170, 333], 2, 2, dim, 16, dtype, new=new, seed=dim + k)
            late_and_large(b, k, 40.0, group)
            check(tok, b, (k, group))


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_tokens_of_many_sizes(tok, dtype):
    """Every token's and group's values of a size of their own, from 2^-25 to 2^25, by one warp and by many."""
    rng = np.random.default_rng(2)
    for lens, dim in (([3000], 128), ([40, 1, 64, 129], 96), ([700] * 40, 64)):
        b = Batch(lens, 1, 3, dim, 16, dtype, seed=5)
        at, g = 16 * pu.groups(dim) * 16, pu.groups(dim)
        words = b.cache[:, 1, :, at:at + 16 * g * 4].copy().view("<u4")
        f = np.float32(2.0) ** rng.integers(-25, 26 if dtype != "float16" else 1, words.shape).astype(np.float32)
        words = pu.bf16_bits(pu.bf16_value(words & 0xFFFF) * f) | pu.bf16_bits(pu.bf16_value(words >> 16) * f) << np.uint32(16)
        b.cache[:, 1, :, at:at + 16 * g * 4] = words.view(np.uint8)
        check(tok, b, dim)


# Long runs: 600 tokens of 16 query heads have 9,600 columns.
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("dim", [64, 96, 200])
def test_long_runs_of_groups_apart(tok, dim, dtype):
    import torch
    for k in (5, 10, 14, 18, 30, 60):
        b = Batch([300, 400], 4, 4, dim, 16, dtype, new=[300, 300], seed=k)
        scale_pairs(b, 1, 20, group=0)
        scale_pairs(b, 1, 20 - k, group=1)
        check(tok, b, k, dtype=torch.float32 if dtype == "float16" else None)
