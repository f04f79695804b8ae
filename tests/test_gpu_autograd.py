"""Derivatives of the embedding lookup on the GPU. Inputs are small whole
numbers, so that every value is exact and equals torch's own indexing."""
import pytest

from tests.ops_util import byte_tokenizer, load

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tok():
    t = byte_tokenizer(load())
    yield t
    t.close()


def inputs(n, rows, dim):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    ids = torch.randint(0, rows, (n,), generator=g, device="cuda", dtype=torch.int32)
    return (ids, *(torch.randint(-2, 3, (m, dim), generator=g, device="cuda").float() for m in (rows, n, rows)))


@pytest.mark.parametrize("n,rows,dim", [(40, 9, 8), (700, 50, 5), (3, 700, 16)])
def test_hessian_products_with_a_tied_table(tok, n, rows, dim):
    """The table is used by the lookup and beside it, as tied output weights are."""
    import torch
    ids, w0, c, v = inputs(n, rows, dim)
    results = []
    for look in (lambda w: tok.embed(ids, w, scale=0.5, skip_id=1),
                 lambda w: torch.where((ids == 1)[:, None], 0.0, w[ids.long()] * 0.5)):
        w = w0.clone().requires_grad_()
        x = look(w)
        (first,) = torch.autograd.grad((x.pow(3) * c).sum() + (x * c).sum() * w.pow(2).sum(), w, create_graph=True)
        (second,) = torch.autograd.grad((first * v).sum(), w)
        results.append((first.detach(), second))
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
    assert float(results[0][1].abs().max()) > 0


def test_embed_grad_is_differentiable(tok):
    import torch
    ids, w, c, _ = inputs(600, 30, 12)
    g = c.to(torch.bfloat16).requires_grad_()
    out = tok.embed_grad(ids, g, 30, scale=2.0, dtype=torch.float32)
    (back,) = torch.autograd.grad((out * w).sum(), g)
    assert back.dtype is torch.bfloat16 and torch.equal(back, (w[ids.long()] * 2).to(torch.bfloat16))


def test_forward_mode(tok):
    import torch
    from torch.autograd import forward_ad
    ids, w, c, v = inputs(700, 50, 8)
    with forward_ad.dual_level():
        value, tangent = forward_ad.unpack_dual(tok.embed(ids, forward_ad.make_dual(w, v), scale=0.5))
        assert torch.equal(value, w[ids.long()] * 0.5) and torch.equal(tangent, v[ids.long()] * 0.5)
        _, tangent = forward_ad.unpack_dual(tok.embed_grad(ids, forward_ad.make_dual(c, c * c), 50))
    assert torch.equal(tangent, torch.zeros_like(w).index_add_(0, ids.long(), c * c))


def test_adjust_logits_raises_where_a_gradient_is_asked_for(tok):
    import torch
    x = torch.randn(3, 900, device="cuda").requires_grad_()
    ids, off = torch.arange(6, dtype=torch.int32, device="cuda"), torch.tensor([0, 2, 4, 6], device="cuda")
    rep = torch.full((3,), 1.5, device="cuda")
    got = tok.adjust_logits(x, prompt=(ids, off), repetition=rep)
    assert torch.equal(got, tok.adjust_logits(x.detach(), prompt=(ids, off), repetition=rep))
    with pytest.raises(RuntimeError, match="no gradient"):
        got.logsumexp(1).sum().backward()
    with pytest.raises(ValueError):
        tok.adjust_logits(x, prompt=(ids, off), repetition=rep, out=torch.empty_like(x))
    with torch.no_grad():
        y = tok.adjust_logits(x, prompt=(ids, off), repetition=rep, out=torch.empty_like(x))
    assert torch.equal(y, got)
