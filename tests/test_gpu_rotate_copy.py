"""Rotations without pairs through the C call: copies, which need no positions
and no table."""
import pytest

from tests.ops_util import byte_tokenizer, load

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim", [1, 2, 4, 6, 8, 64, 101])
@pytest.mark.parametrize("kind,out_kind", [("float32", "float32"), ("bfloat16", "bfloat16"), ("float16", "float32")])
def test_no_pairs_no_positions(dim, kind, out_kind, interleaved):
    import torch
    bpe = load()
    tok = byte_tokenizer(bpe)
    x = torch.randn(7, 3, dim, device="cuda").to(getattr(torch, kind))
    out = torch.zeros(7, 3, dim, dtype=getattr(torch, out_kind), device="cuda")
    codes = {"float32": bpe.F32, "float16": bpe.F16, "bfloat16": bpe.BF16}
    bpe.bpe_rotate(tok.handle, x.data_ptr(), codes[kind], 7, 3, dim, 3 * dim, dim, None, None, 0, interleaved, False,
                   2.0, out.data_ptr(), codes[out_kind], 3 * dim, dim, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(out, x.to(out.dtype))
    tok.close()
