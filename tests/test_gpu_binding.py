"""Arguments at the edge of what the operators around the model take, on the GPU."""
import pytest

from tests.ops_util import byte_tokenizer, load

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bpe():
    return load()


@pytest.fixture(scope="module")
def tok(bpe):
    t = byte_tokenizer(bpe)
    yield t
    t.close()


def status(bpe, tok):
    import torch
    try:
        bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)
    except bpe.BpeError as e:
        return e.code
    return 0


def test_masks_without_rows(bpe, tok):
    import torch
    x, none = torch.randn(3, 100, device="cuda"), torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(bpe.BpeError):
        tok.adjust_logits(x, mask=none)
    rows = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    assert torch.equal(tok.adjust_logits(x, mask=none, mask_rows=rows), x) and status(bpe, tok) == 0
    rows[1] = 0  # a mask that is not there: reported, not taken as one that allows everything
    assert torch.equal(tok.adjust_logits(x, mask=none, mask_rows=rows), x) and status(bpe, tok) == 7
    with pytest.raises(ValueError):
        tok.adjust_logits(x, mask_rows=rows)
