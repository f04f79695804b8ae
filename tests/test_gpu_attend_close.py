"""Attention within bounds that count its roundings (paged_close.py): a scale
that is a tenth off, equal weights, a token too many or too few do not pass."""
import numpy as np
import pytest

from tests.ops_util import byte_tokenizer, load
from tests.paged_close import check, scale_pairs
from tests.test_gpu_attend import Batch

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "float16", "bfloat16"]


@pytest.fixture(scope="module")
def tok():
    t = byte_tokenizer(load())
    yield t
    t.close()


def last_tokens_count(b):
    """The last token of each request, and of those that new ones see, has values 16 times the others'."""
    for r, length in enumerate(b.lens):
        for t in range(max(0, int(length) - 2), int(length)):
            scale_pairs(b, 1, 4, r, t)
    return b


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [1, 8, 21, 32, 40, 64, 72, 96, 128, 130, 160, 192, 200, 256])
def test_dims(tok, dim, dtype):
    check(tok, Batch([1, 33, 70, 640], 2, 3, dim, 16, dtype, seed=dim))


@pytest.mark.parametrize("heads,group", [(1, 1), (3, 2), (2, 5), (1, 8), (2, 9), (1, 16), (1, 17), (5, 1), (1, 40)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_head_layouts(tok, heads, group, dtype):
    check(tok, Batch([37, 1, 64, 5, 300], heads, group, 64, 8, dtype, seed=group))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("block", [1, 3, 16, 31, 33, 100, 256])
def test_blocks_and_lengths(tok, block, dtype):
    check(tok, last_tokens_count(Batch([0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 200], 1, 2, 128, block, dtype,
                                       seed=block)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[5000], [20_000], [1, 4000, 2, 3, 900], [100] * 300, list(range(1, 200))])
def test_lengths(tok, lens, dtype):
    check(tok, last_tokens_count(Batch(lens, 2, 2, 32, 16, dtype, seed=len(lens))))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,group,dim", [(2, 4, 64), (1, 1, 128), (2, 3, 40), (1, 16, 256)])
def test_new_tokens(tok, heads, group, dim, dtype):
    b = Batch([40, 9, 5, 64, 200, 70, 0], heads, group, dim, 16, dtype, new=[1, 0, 5, 33, 2, 70, 0], pad=4, seed=group)
    check(tok, b)


@pytest.mark.parametrize("dtype,heads,group,dim,block", [
    ("bfloat16", 16, 1, 128, 16), ("float16", 4, 4, 64, 16), ("bfloat16", 8, 2, 21, 3), ("float16", 8, 3, 96, 100),
    ("bfloat16", 4, 5, 200, 16), ("float16", 16, 1, 256, 7), ("bfloat16", 4, 8, 32, 1), ("bfloat16", 8, 2, 130, 32),
    ("float16", 16, 8, 128, 16), ("bfloat16", 16, 8, 96, 16)])
def test_long_runs(tok, dtype, heads, group, dim, block):
    b = Batch([128, 500, 300, 700, 131, 9, 400], heads, group, dim, block, dtype, new=[128, 1, 300, 64, 129, 0, 16],
              pad=3, seed=dim)
    check(tok, b)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_long_runs_far_behind(tok, dtype):
    """Behind 3,000 tokens, so that a tile of columns is scaled often; results in 32 bits show its own roundings."""
    import torch
    check(tok, Batch([3200, 3130], 16, 2, 64, 16, dtype, new=[200, 130], seed=9), dtype=torch.float32)


@pytest.mark.parametrize("scale", [1.0, 0.0, -0.4, 0.01])
@pytest.mark.parametrize("dtype", DTYPES)
def test_scales(tok, scale, dtype):
    check(tok, Batch([90, 40], 1, 3, 64, 16, dtype, seed=7), scale, scale=scale)
    check(tok, Batch([200, 330], 16, 1, 64, 16, dtype, new=[200, 330], seed=21), scale, scale=scale)


@pytest.mark.parametrize("dtype", DTYPES)
def test_sharp_scores(tok, dtype):
    for by in (6.0, 15.0):
        check(tok, Batch([3000, 200], 1, 2, 64, 16, dtype, seed=11, by=by), by)
        check(tok, Batch([600, 200], 16, 1, 64, 16, dtype, new=[330, 190], seed=22, by=by), by)


@pytest.mark.parametrize("dtype,out", [("float32", "bfloat16"), ("bfloat16", "float32"), ("float16", "bfloat16"),
                                       ("bfloat16", "float16"), ("float16", "float32")])
def test_result_types(tok, dtype, out):
    import torch
    check(tok, Batch([50, 3, 900], 1, 4, 64, 16, dtype), dtype=getattr(torch, out))
