"""What the binding of the operators around the model refuses or hands to the
library, on the host (see cpu_ops)."""
import pytest

from tests.cpu_ops import tokenizer


@pytest.fixture()
def tok(monkeypatch):
    return tokenizer(monkeypatch)


@pytest.fixture(scope="module")
def bpe():
    import byte_level_bpe_pretokenize_gb300 as m
    return m


def test_masks_without_rows(bpe, tok):
    """An empty table of masks has no address; it must not pass for no mask at all."""
    import torch
    x, none = torch.ones(2, 40), torch.zeros(0, 2, dtype=torch.int32)
    with pytest.raises(bpe.BpeError, match="fewer masks than rows") as e:
        tok.adjust_logits(x, mask=none)
    assert e.value.code == 1 and not tok._lib.calls
    rows = torch.tensor([-1, 0], dtype=torch.int32)
    tok.adjust_logits(x, mask=none, mask_rows=rows)
    args = tok._lib.logits_args
    assert args.mask and args.n_masks == 0 and args.mask_rows == rows.data_ptr()
    assert tok.adjust_logits(torch.ones(0, 40), mask=none).shape == (0, 40)


def test_mask_rows_need_masks(tok):
    import torch
    with pytest.raises(ValueError, match="no mask"):
        tok.adjust_logits(torch.ones(2, 40), mask_rows=torch.zeros(2, dtype=torch.int32))


def test_dtype_and_out_must_agree(tok):
    import torch
    ids, w, x = torch.zeros(3, dtype=torch.int32), torch.ones(5, 4), torch.ones(3, 4)
    for call, out in ((lambda **k: tok.embed(ids, w, **k), torch.zeros(3, 4)),
                      (lambda **k: tok.embed_grad(ids, x, 5, **k), torch.zeros(5, 4)),
                      (lambda **k: tok.adjust_logits(x, **k), torch.zeros(3, 4))):
        with pytest.raises(ValueError, match="dtype"):
            call(out=out, dtype=torch.bfloat16)
        assert not tok._lib.calls
        assert call(out=out, dtype=torch.float32) is out and len(tok._lib.calls) == 1
        tok._lib.calls.clear()


def test_skip_id_is_not_cut_to_32_bits(tok):
    import torch
    ids, w, x = torch.tensor([1, 2, 3], dtype=torch.int32), torch.ones(5, 4), torch.ones(3, 4)
    for skip in (2 ** 32 + 2, 2 ** 31, -2 ** 31 - 1, -2 ** 32 + 2):
        with pytest.raises(ValueError, match="skip_id"):
            tok.embed(ids, w, skip_id=skip)
        with pytest.raises(ValueError, match="skip_id"):
            tok.embed_grad(ids, x, 5, skip_id=skip)
    assert tok.embed(ids, w, skip_id=2).sum(1).tolist() == [4, 0, 4]
    assert tok.embed(ids, w, skip_id=-2 ** 31).sum(1).tolist() == tok.embed(ids, w).sum(1).tolist() == [4, 4, 4]
