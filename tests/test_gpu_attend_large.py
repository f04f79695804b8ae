"""Attention over values next to the largest floats: results are means, so they
are finite, also where several workers have a share of the sums."""
import pytest

from tests.ops_util import byte_tokenizer, load
from tests.paged_close import check, scale_pairs
from tests.test_gpu_attend import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("lens,new", [([30], None), ([20_000], None), ([300] * 30, None), ([5000, 3], [3, 1]),
                                      ([300, 290], [300, 230])])
@pytest.mark.parametrize("exponent", [60, 100, 124])
def test_large_values(exponent, lens, new, dtype):
    tok = byte_tokenizer(load())
    b = Batch(lens, 16 if new and new[0] > 200 else 2, 1, 64, 16, dtype, new=new, seed=exponent)
    scale_pairs(b, 1, exponent)
    check(tok, b)
    tok.close()
