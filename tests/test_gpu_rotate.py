"""Rotary positions on the GPU against rotations in 64 bits, and their
gradients."""
import numpy as np
import pytest

from tests.ops_util import assert_close, byte_tokenizer, load
from tests.paged_util import turned

pytestmark = pytest.mark.gpu

TYPES = ["float32", "float16", "bfloat16"]


@pytest.fixture(scope="module")
def tok():
    t = byte_tokenizer(load())
    yield t
    t.close()


def frequencies(dim, base=10_000.0):
    return base ** (-np.arange(0, dim, 2) / dim)


def inputs(tokens, heads, dim, dtype, seed=0, far=5000):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(tokens, heads, dim, generator=g, device="cuda").to(getattr(torch, dtype))
    p = torch.randint(0, far, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    return x, p


def check(got, x, p, part, interleaved, scale=1.0, inverse=False, f=None, label=""):
    import torch
    f = frequencies(part) if f is None else f
    want, bound = turned(x.double().cpu().numpy(), p.cpu().numpy(), f, interleaved, scale, inverse)
    assert_close(got, torch.from_numpy(want), torch.from_numpy(bound), label)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,heads,dim,part", [
    (1, 1, 2, 2), (3, 5, 128, 128), (7, 3, 80, 50), (65, 2, 96, 24), (4, 9, 64, 0), (300, 4, 21, 20), (2, 40, 128, 128),
    (5, 3, 72, 72), (1000, 1, 16, 4), (2, 1, 260, 258), (1, 1, 1, 0), (6, 70, 100, 100)])
def test_rotations(tok, tokens, heads, dim, part, dtype, interleaved):
    x, p = inputs(tokens, heads, dim, dtype)
    table = tok.rotary_table(part)
    check(tok.rotate(x, p, table, interleaved), x, p, part, interleaved)
    check(tok.rotate(x, p, table, interleaved, scale=1.25, inverse=True), x, p, part, interleaved, 1.25, True)


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_types(tok, dtype, out):
    import torch
    x, p = inputs(33, 3, 64, dtype)
    got = tok.rotate(x, p, tok.rotary_table(64), dtype=getattr(torch, out))
    assert got.dtype is getattr(torch, out)
    check(got, x, p, 64, False)


def test_far_positions(tok):
    """Positions at which a 32-bit angle would be off by radians, and every int32."""
    import torch
    x, _ = inputs(9, 2, 64, "float32")
    p = torch.tensor([0, 1, 2 ** 20 + 1, 10 ** 7, 2 ** 31 - 1, -1, -(2 ** 31), -12345, 99_999_999], dtype=torch.int32,
                     device="cuda")
    f = frequencies(64)
    # the reference's own angle is off by half a step of a 64-bit number of p f radians, as is each frequency in turns
    want, bound = turned(x.double().cpu().numpy(), p.cpu().numpy(), f, False, 1.0)
    slack = np.abs(p.cpu().numpy().astype(np.float64))[:, None, None] * 4 * 2.0 ** -53
    bound += slack * np.abs(x.double().cpu().numpy()).max() * 2
    assert_close(tok.rotate(x, p, tok.rotary_table(64)), torch.from_numpy(want), torch.from_numpy(bound))


@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_and_in_place(tok, interleaved):
    import torch
    fused, p = inputs(50, 1, 12 * 64 + 3, "bfloat16")
    table = tok.rotary_table(48)
    for start in (0, 1, 3):  # aligned and odd addresses
        x = fused[:, 0, start:start + 10 * 64].unflatten(1, (10, 64))
        want = tok.rotate(x.contiguous(), p, table, interleaved)
        assert torch.equal(tok.rotate(x, p, table, interleaved), want)
        whole = fused.clone()
        y = whole[:, 0, start:start + 10 * 64].unflatten(1, (10, 64))
        assert tok.rotate(y, p, table, interleaved, out=y) is y
        assert torch.equal(y, want)
        left = torch.ones(whole.shape[2], dtype=torch.bool, device="cuda")
        left[start:start + 10 * 64] = False
        assert torch.equal(whole[..., left], fused[..., left])
    # heads before tokens, one token for all, one head for all
    x, p = inputs(20, 6, 64, "float16")
    want = tok.rotate(x, p, table, interleaved)
    assert torch.equal(tok.rotate(x.transpose(0, 1).contiguous().transpose(0, 1), p, table, interleaved), want)
    out = torch.empty(6, 20, 64, dtype=torch.float16, device="cuda").transpose(0, 1)
    assert torch.equal(tok.rotate(x, p, table, interleaved, out=out), want)
    for y in (x[:1].expand(20, 6, 64), x[:, :1].expand(20, 6, 64)):
        assert torch.equal(tok.rotate(y, p, table, interleaved), tok.rotate(y.contiguous(), p, table, interleaved))
    assert torch.equal(tok.rotate(x[..., ::2], p, tok.rotary_table(32), interleaved),
                       tok.rotate(x[..., ::2].contiguous(), p, tok.rotary_table(32), interleaved))


@pytest.mark.parametrize("interleaved", [False, True])
def test_infinities_stay_in_their_pairs(tok, interleaved):
    import torch
    x, p = inputs(3, 2, 40, "float32")
    x[0, 0, 30], x[1, 1, 39], x[2, 0, 5] = float("inf"), float("nan"), float("inf")
    y = tok.rotate(x, p, tok.rotary_table(24), interleaved)
    assert y[0, 0, 30] == float("inf") and y[1, 1, 39].isnan()  # behind the turned part: copied
    wrong = ~y.isfinite()
    pair = (4, 5) if interleaved else (5, 17)
    assert wrong.nonzero().tolist() == sorted([[0, 0, 30], [1, 1, 39]] + [[2, 0, e] for e in pair if wrong[2, 0, e]])
    assert wrong[2, 0, pair[0]] or wrong[2, 0, pair[1]]


def test_scaled_tables(tok):
    f = frequencies(64)
    turns = 8192 * f / (2 * np.pi)
    keep = np.clip((turns - 1) / 3, 0, 1)
    x, p = inputs(40, 2, 64, "float32", far=131_072)
    by_parts = f * (keep + (1 - keep) / 16)
    check(tok.rotate(x, p, tok.rotary_table(64, factor=16.0, original=8192)), x, p, 64, False, f=by_parts)
    check(tok.rotate(x, p, tok.rotary_table(64, factor=4.0)), x, p, 64, False, f=f / 4)
    odd = np.linspace(-2.0, 9.0, 32)
    check(tok.rotate(x, p, tok.rotary_table(64, frequencies=odd)), x, p, 64, False, f=odd)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_gradient(tok, dtype, interleaved):
    """Backward is the transposed rotation: against its formula in 64 bits, and <R x, g> = <x, R' g>."""
    import torch
    x, p = inputs(30, 4, 72, dtype)
    g, _ = inputs(30, 4, 72, dtype, seed=1)
    x.requires_grad_()
    table = tok.rotary_table(50)
    y = tok.rotate(x, p, table, interleaved, scale=1.5)
    (grad,) = torch.autograd.grad(y, x, g)
    assert grad.dtype is x.dtype
    check(grad, g, p, 50, interleaved, 1.5, True)
    wide = x.detach().double(), g.double()
    left, right = (y.detach().double() * wide[1]).sum(), (wide[0] * grad.double()).sum()
    # each side rounds every element by half a step of its type
    u = torch.finfo(x.dtype).eps / 2 + 16 * 2.0 ** -24
    assert abs(float(left - right)) <= 2 * u * 3 * float((wide[0].abs() * wide[1].abs()).sum() * 1.5 +
                                                         wide[0].norm() * wide[1].norm() * 1.5)


def test_gradient_by_differences(tok):
    """The map is linear, so a difference quotient has no error but rounding: steps of 1 on whole numbers."""
    import torch
    x, p = inputs(3, 2, 16, "float32")
    table = tok.rotary_table(12)
    c, _ = inputs(3, 2, 16, "float32", seed=4)
    x = x.requires_grad_()
    (grad,) = torch.autograd.grad((tok.rotate(x, p, table) * c).sum(), x)
    base = tok.rotate(x.detach(), p, table).double()
    for at in np.ndindex(3, 2, 16):
        moved = x.detach().clone()
        moved[at] += 1
        difference = ((tok.rotate(moved, p, table).double() - base) * c.double()).sum()
        # two rounded rotations of a pair below 8, times c below 5
        assert abs(float(difference) - float(grad[at])) <= 2 * 2 * 8 * 5 * 12 * 2.0 ** -24


def test_derivatives_of_higher_order_and_forward_mode(tok):
    import torch
    from torch.autograd import forward_ad
    x, p = inputs(10, 2, 32, "float32")
    v, _ = inputs(10, 2, 32, "float32", seed=2)
    table = tok.rotary_table(32)
    x.requires_grad_()
    y = tok.rotate(x, p, table)
    (first,) = torch.autograd.grad(y.pow(3).sum(), x, create_graph=True)
    (second,) = torch.autograd.grad((first * v).sum(), x)
    want = tok.rotate(6 * y.detach() * tok.rotate(v, p, table), p, table, inverse=True)
    assert float((second - want).abs().max()) <= 1e-5 * float(want.abs().max())
    with forward_ad.dual_level():
        value, tangent = forward_ad.unpack_dual(tok.rotate(forward_ad.make_dual(x.detach(), v), p, table))
    assert torch.equal(value, y.detach()) and torch.equal(tangent, tok.rotate(v, p, table))


def test_gradient_of_a_broadcast_input(tok):
    import torch
    x, p = inputs(20, 1, 32, "float32")
    x.requires_grad_()
    table = tok.rotary_table(32)
    (grad,) = torch.autograd.grad(tok.rotate(x.expand(20, 8, 32), p, table).sum(), x)
    ones = tok.rotate(torch.ones(20, 8, 32, device="cuda"), p, table, inverse=True)
    assert grad.shape == x.shape and float((grad - ones.sum(1, keepdim=True)).abs().max()) <= 1e-5 * 8


def test_empty(tok):
    import torch
    table, none = tok.rotary_table(8), torch.zeros(0, dtype=torch.int32, device="cuda")
    assert tok.rotate(torch.zeros(0, 3, 8, device="cuda"), none, table).shape == (0, 3, 8)
    assert tok.rotate(torch.zeros(0, 0, 8, device="cuda"), none, table).shape == (0, 0, 8)
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert tok.rotate(torch.zeros(2, 0, 8, device="cuda"), zero, table).shape == (2, 0, 8)


def test_captured_forward_and_backward(tok):
    """A training step's graph with an eager graph of the same leaf alive."""
    import torch
    x, p = inputs(64, 4, 64, "bfloat16")
    g, _ = inputs(64, 4, 64, "bfloat16", seed=3)
    table = tok.rotary_table(64)
    want = torch.autograd.grad(tok.rotate(x.requires_grad_(), p, table), x, g)[0]
    x = x.detach()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = tok.rotate(x, p, table)
        back = tok.rotate(g, p, table, inverse=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = tok.rotate(x, p, table)
        back = tok.rotate(g, p, table, inverse=True)
    y.zero_(), back.zero_()
    graph.replay()
    assert torch.equal(y, tok.rotate(x, p, table)) and torch.equal(back, want)


def test_a_captured_training_step(tok):
    """Forward and backward through autograd in one graph, replayed on new inputs."""
    import torch
    x, p = inputs(64, 4, 64, "float32")
    g, _ = inputs(64, 4, 64, "float32", seed=3)
    table = tok.rotary_table(64)
    x.requires_grad_()

    def step():
        y = tok.rotate(x, p, table, scale=1.5)
        (grad,) = torch.autograd.grad((y * g).sum(), x)
        return grad

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grad = step()
    for seed in (5, 6):
        g.copy_(inputs(64, 4, 64, "float32", seed=seed)[0])
        p.copy_(inputs(64, 1, 1, "float32", seed=seed)[1])
        graph.replay()
        assert torch.equal(grad, tok.rotate(g, p, table, scale=1.5, inverse=True))


def test_refusals(tok):
    import torch

    import byte_level_bpe_pretokenize_gb300 as bpe
    x, p = inputs(4, 2, 16, "float32")
    table = tok.rotary_table(16)
    for bad in (lambda: tok.rotate(x.double(), p, table), lambda: tok.rotate(x[0], p, table),
                lambda: tok.rotate(x, p.long(), table), lambda: tok.rotate(x, p[:3], table),
                lambda: tok.rotate(x.cpu(), p, table), lambda: tok.rotate(x, p, tok.rotary_table(18)),
                lambda: tok.rotate(x, p, table, out=torch.empty(4, 2, 15, device="cuda")),
                lambda: tok.rotate(x, p, table, out=torch.empty(4, 2, 16, device="cuda"), dtype=torch.float16),
                lambda: tok.rotate(x.clone().requires_grad_(), p, table, out=torch.empty_like(x)),
                lambda: tok.rotary_table(7), lambda: tok.rotary_table(8, frequencies=[1.0])):
        with pytest.raises(ValueError):
            bad()
    row = torch.zeros(2, 16, device="cuda").expand(4, 2, 16)
    with pytest.raises(bpe.BpeError, match="overlap"):
        tok.rotate(x, p, table, out=row)
    with pytest.raises(bpe.BpeError, match="in place"):
        tok.rotate(x, p, table, out=x.as_strided((4, 2, 16), (16, 64, 1)))
