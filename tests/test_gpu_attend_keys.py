"""Long runs over keys of very different sizes: what halves do not hold in one
unit is computed as short runs are."""
import pytest

from tests.ops_util import byte_tokenizer, load
from tests.paged_close import check, scale_pairs
from tests.test_gpu_attend import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tok():
    t = byte_tokenizer(load())
    yield t
    t.close()


# 600 tokens of 16 query heads have 9,600 columns
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("dim", [64, 96, 200])
def test_long_runs_of_keys_apart(tok, dim, dtype):
    """A group of keys 2^k larger, which queries do not ask for, leaves the others their scores."""
    for k in (5, 10, 14, 18, 24, 30):
        b = Batch([300, 400], 4, 4, dim, 16, dtype, new=[300, 300], seed=k)
        scale_pairs(b, 0, k, group=0)
        b.q[..., :32] = 0
        check(tok, b, k)
