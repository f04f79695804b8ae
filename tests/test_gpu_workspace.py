"""The handle's workspace: what a call needs never grows as the call gets
smaller, so that one call of the largest size makes room for all others."""
import pytest

from tests.ops_util import byte_tokenizer, load

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bpe():
    return load()


@pytest.fixture()
def tok(bpe):
    """A handle of its own for each test: none has a workspace yet."""
    t = byte_tokenizer(bpe)
    yield t
    t.close()


def gradient(tok, n, rows, dim):
    import torch
    ids = (torch.arange(n, device="cuda") * 7919 % rows).to(torch.int32)
    grad = torch.ones(n, dim, dtype=torch.bfloat16, device="cuda")
    return tok.embed_grad(ids, grad, rows)


def test_up_to_512_tokens_take_none(bpe, tok):
    for n in (0, 1, 300, 512):
        gradient(tok, n, 5000, 1024)
    assert bpe.bpe_workspace_bytes(tok.handle) == 0


@pytest.mark.parametrize("n,dim", [(4864, 4096), (2432, 8192), (20_000, 1000), (70_000, 512)])
def test_a_smaller_gradient_needs_no_more(bpe, tok, n, dim):
    rows = 900
    gradient(tok, n, rows, dim)
    held = bpe.bpe_workspace_bytes(tok.handle)
    assert held > 0
    for fewer in (n - 1, n * 3 // 4, n // 2 + 1, n // 2, 2047, 1025, 600, 513, 512, 17, 1):
        for columns in (dim, dim - 1, dim * 2 // 3, 513, 512, 511, 64, 1):
            gradient(tok, min(fewer, n), rows, min(columns, dim))
            assert bpe.bpe_workspace_bytes(tok.handle) == held, (fewer, columns)
