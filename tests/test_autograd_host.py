"""Derivatives through the binding of the operators around the model, on the
host (the library's calls by numpy): every order against torch's own indexing,
or an error, never a number that lacks a term. Inputs are small whole numbers,
so that every value is exact."""
import pytest

from tests.cpu_ops import tokenizer

ROWS, DIM, SCALE, SKIP = 7, 3, 0.5, 2


@pytest.fixture()
def tok(monkeypatch):
    return tokenizer(monkeypatch)


def inputs(seed=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, ROWS, (11,), generator=g, dtype=torch.int32)
    return (ids, torch.randint(-3, 4, (ROWS, DIM), generator=g).float(),
            torch.randint(-3, 4, (11, DIM), generator=g).float(), torch.randint(-3, 4, (ROWS, DIM), generator=g).float())


def plain_embed(ids, weight):
    import torch
    return torch.where((ids == SKIP)[:, None], 0.0, weight[ids.long()] * SCALE)


def embed(tok, ids, weight):
    return tok.embed(ids, weight, scale=SCALE, skip_id=SKIP)


def tied_loss(x, weight, c):
    """A loss that is of third order in the table, through the lookup and beside it."""
    return ((x * x) * c).sum() + (x @ weight.t()).pow(2).sum() + weight.pow(3).sum()


@pytest.mark.parametrize("tied", [False, True])
def test_second_and_third_derivatives(tok, tied):
    import torch
    ids, w0, c, v = inputs()
    results = []
    for look in (lambda w: embed(tok, ids, w), lambda w: plain_embed(ids, w)):
        w = w0.clone().requires_grad_()
        x = look(w)
        loss = tied_loss(x, w, c) if tied else (x.pow(4) * c).sum()
        (first,) = torch.autograd.grad(loss, w, create_graph=True)
        (second,) = torch.autograd.grad((first * v).sum(), w, create_graph=True)  # the Hessian's product with v
        (third,) = torch.autograd.grad((second * v).sum(), w)
        results.append((x.detach(), first.detach(), second.detach(), third))
    for name, got, want in zip(("value", "first", "second", "third"), *results):
        assert torch.equal(got, want), name
    assert tok._lib.calls.count("embed") >= 2 and tok._lib.calls.count("embed_grad") >= 2


def test_gradient_penalty(tok):
    """A penalty on the upstream gradient's image: a loss of embed_grad's result alone."""
    import torch
    ids, w0, c, _ = inputs(1)
    results = []
    for look in (lambda w: embed(tok, ids, w), lambda w: plain_embed(ids, w)):
        w, u = w0.clone().requires_grad_(), c.clone().requires_grad_()
        (first,) = torch.autograd.grad((look(w) * u * u).sum(), w, create_graph=True)
        results.append(torch.autograd.grad(first.pow(2).sum(), u)[0])
    assert torch.equal(*results)


def test_embed_grad_is_differentiable(tok):
    import torch
    ids, _, c, v = inputs(2)
    g = c.clone().requires_grad_()
    out = tok.embed_grad(ids, g, ROWS, scale=SCALE, skip_id=SKIP)
    (back,) = torch.autograd.grad((out * v).sum(), g)
    assert torch.equal(back, plain_embed(ids, v))
    with torch.no_grad():
        assert not tok.embed_grad(ids, g, ROWS).requires_grad
    assert not tok.embed_grad(ids, g, ROWS, out=torch.zeros(ROWS, DIM)).requires_grad


def test_forward_mode(tok):
    import torch
    from torch.autograd import forward_ad
    ids, w, c, v = inputs(3)
    with forward_ad.dual_level(), torch.no_grad():
        value, tangent = forward_ad.unpack_dual(embed(tok, ids, forward_ad.make_dual(w, v)))
        assert torch.equal(value, plain_embed(ids, w)) and torch.equal(tangent, plain_embed(ids, v))
        g = forward_ad.make_dual(c, c * c)
        value, tangent = forward_ad.unpack_dual(tok.embed_grad(ids, g, ROWS, scale=SCALE))
        assert torch.equal(value, tok.embed_grad(ids, c, ROWS, scale=SCALE))
        assert torch.equal(tangent, tok.embed_grad(ids, c * c, ROWS, scale=SCALE))
    with forward_ad.dual_level():
        assert forward_ad.unpack_dual(embed(tok, ids, w)).tangent is None  # not a dual tensor


def test_forward_over_reverse(tok):
    import torch
    from torch.autograd import forward_ad
    ids, w0, c, v = inputs(4)
    results = []
    for look in (lambda w: embed(tok, ids, w), lambda w: plain_embed(ids, w)):
        with forward_ad.dual_level():
            w = forward_ad.make_dual(w0.clone().requires_grad_(), v)
            (first,) = torch.autograd.grad(tied_loss(look(w), w, c), w, create_graph=True)
            value, tangent = forward_ad.unpack_dual(first)
            results.append((value.detach(), tangent.detach()))
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])


def test_adjust_logits_is_not_cut_off_silently(tok):
    import torch
    from torch.autograd import forward_ad
    x = torch.ones(2, 5)
    f = torch.ones(2)
    bias = (torch.zeros(1, dtype=torch.int32), torch.ones(1), torch.tensor([0, 1, 1]))
    cases = [(x.clone().requires_grad_(), {})]
    cases += [(x, {name: f.clone().requires_grad_()}) for name in ("repetition", "frequency", "presence")]
    cases += [(x, {"bias": (bias[0], bias[1].clone().requires_grad_(), bias[2])})]
    for logits, more in cases:
        got = tok.adjust_logits(logits, **more)
        assert torch.equal(got, x * 0.5)  # the value is there, to sample from
        with pytest.raises(RuntimeError, match="no gradient"):
            got.sum().backward()
        with pytest.raises(ValueError, match="derivative"):
            tok.adjust_logits(logits, out=torch.zeros(2, 5), **more)
        with torch.no_grad():
            assert not tok.adjust_logits(logits, **more).requires_grad
            tok.adjust_logits(logits.detach().clone(), out=torch.zeros(2, 5), **more)
    with forward_ad.dual_level():
        with pytest.raises(RuntimeError):
            tok.adjust_logits(forward_ad.make_dual(x, x))
    assert not tok.adjust_logits(x, repetition=f, bias=bias).requires_grad


def test_what_is_written_counts_as_written(tok, monkeypatch):
    """A backward pass through a tensor that a call has since overwritten raises, as torch's own writes make it."""
    import torch

    import byte_level_bpe_pretokenize_gb300 as bpe
    ids, w0, c, _ = inputs(5)
    i32 = dict(dtype=torch.int32)
    monkeypatch.setattr(bpe, "bpe_encode_batch", lambda *a: None)
    monkeypatch.setattr(bpe.Tokenizer, "_stream", staticmethod(lambda: 0))
    tok._lib.bpe_plan_blocks = lambda *a: 0
    table = torch.zeros(2, 3, **i32)

    logits = torch.ones(2, 4)
    rows, grad = torch.zeros(11, DIM), torch.zeros(ROWS, DIM)
    for saved, write in ((logits, lambda: tok.adjust_logits(logits, out=logits)),
                         (rows, lambda: tok.embed(ids, w0, out=rows)),
                         (grad, lambda: tok.embed_grad(ids, c, ROWS, out=grad)),
                         (grad, lambda: tok.embed_grad(ids, c, ROWS, out=grad, accumulate=True))):
        one = torch.ones_like(saved).requires_grad_()
        loss = (saved * one).sum()  # saves what is written below
        with torch.no_grad():
            write()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    # the next batch's ids in the buffer of this one's
    w = w0.clone().requires_grad_()
    loss = embed(tok, ids, w).sum()
    tok.encode_into(torch.zeros(3, dtype=torch.uint8), torch.zeros(2, dtype=torch.int64), ids,
                    torch.zeros(2, dtype=torch.int64), False)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    before = table._version
    tok.plan_blocks(None, None, table, torch.zeros(4, **i32), 16)
    assert table._version > before


def test_out_must_not_require_a_gradient(tok):
    import torch
    ids, w, c, _ = inputs(6)
    hidden = torch.zeros(11, DIM).requires_grad_() * 1
    with pytest.raises(ValueError, match="require a gradient"):
        tok.embed(ids, w, out=hidden)
    with pytest.raises(ValueError, match="require a gradient"):
        tok.embed_grad(ids, c, ROWS, out=torch.zeros(ROWS, DIM).requires_grad_())
    with pytest.raises(ValueError, match="require a gradient"):
        tok.adjust_logits(c, out=hidden)
    table = torch.zeros(ROWS, DIM).requires_grad_()
    with torch.no_grad():  # an update by hand
        tok.embed_grad(ids, c, ROWS, out=table)
    assert torch.equal(table, tok.embed_grad(ids, c, ROWS))
    with torch.inference_mode():
        tok.embed(ids, w, out=torch.zeros(11, DIM))
        tok.adjust_logits(c, out=hidden.detach())
