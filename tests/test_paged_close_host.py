"""The bound of attention in paged_close.py, on the host: it is a small part of
the results, and results of a wrong scale, of equal weights, of a token too many
or too few, and zeros lie outside of it. The mistakes are made in the oracle."""
import numpy as np
import pytest

from tests import paged_close as pc
from tests import paged_util as pu
from tests.ops_util import ROUNDOFF
from tests.test_gpu_attend import Batch

DTYPES = ["float32", "float16", "bfloat16"]


def oracle(b, lens=None, **k):
    parts = 2 if "32" in str(b.q.dtype) else 1
    return pc.attention(b.q.double().numpy(), b.cache, b.table, b.lens if lens is None else lens, b.block, b.offsets,
                        parts=parts, **k)


def outside(b, wrong):
    """The part of the results that would be off."""
    want, bound = oracle(b)
    u = ROUNDOFF[str(b.q.dtype).replace("torch.", "")]
    real = ~np.isnan(want)
    return float((np.abs(wrong - want) > bound + u * (np.abs(want) + bound))[real].mean())


def batches(dtype):
    for dim in (32, 64, 128, 200, 256):
        yield Batch([1, 33, 70], 2, 3, dim, 16, dtype, seed=dim)
    yield Batch([1000, 300], 2, 2, 128, 16, dtype, seed=1)
    yield Batch([128, 500, 300], 2, 2, 64, 16, dtype, new=[128, 1, 300], seed=1)
    yield Batch([300, 290], 16, 1, 32, 16, dtype, new=[300, 250], seed=1)  # a long run


@pytest.mark.parametrize("dtype", DTYPES)
def test_wrong_results_lie_outside(dtype):
    for b in batches(dtype):
        right = b.dim ** -0.5
        for by in (0.9, 1.1, 0.0):
            assert outside(b, oracle(b, scale=right * by)[0]) > 0.3
        if dtype == "float32":
            assert outside(b, oracle(b, scale=right * 1.01)[0]) > 0.3
        assert outside(b, oracle(b, np.maximum(b.lens - 1, 0))[0]) > 0.05  # sees one token less
        assert outside(b, np.zeros(b.q.shape)) > 0.9
        assert outside(b, oracle(b)[0]) == 0.0


@pytest.mark.parametrize("dtype", DTYPES)
def test_the_bound_is_small(dtype):
    for b in batches(dtype):
        want, bound = oracle(b)
        real = ~np.isnan(want)
        assert np.sqrt((bound[real] ** 2).mean()) < (0.002 if dtype == "float32" else 0.02) * np.sqrt((want[real] ** 2).mean())


@pytest.mark.parametrize("dtype", DTYPES)
def test_it_agrees_with_the_other_oracle(dtype):
    for b in batches(dtype):
        want, _ = oracle(b)
        other, _ = pu.attention(b.q.double().numpy(), b.cache, b.table, b.lens, b.block, b.offsets)
        assert np.array_equal(np.isnan(want), np.isnan(other))
        assert np.nanmax(np.abs(want - other)) < 1e-12
