"""Embedding lookup and its gradient against 64-bit computations.

Bounds. Lookup: one 32-bit product (relative error 2^-24) and one rounding to
the output's type. Gradient of a row with m tokens: at most m - 1 additions and
one product in 32 bits, each with a relative error of at most 2^-24 of the sum
of magnitudes, so (m + 1) 2^-24 (1 + small) scale sum|x|, one more addition when
accumulating, and one rounding to the output's type.
"""
import pytest

from tests.ops_util import assert_close, byte_tokenizer, load

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def bpe():
    return load()


@pytest.fixture(scope="module")
def tok(bpe):
    t = byte_tokenizer(bpe)
    yield t
    t.close()


def dtypes():
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rand(shape, dtype, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtypes()[dtype])


def make_ids(n, rows, kind, seed=0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + n)
    if kind == "uniform":
        return torch.randint(0, rows, (n,), generator=g, device="cuda", dtype=torch.int32)
    if kind == "one":
        return torch.full((n,), rows // 2, dtype=torch.int32, device="cuda")
    if kind == "down":
        return (rows - 1 - torch.arange(n, device="cuda") % rows).to(torch.int32)
    # skewed: a few rows take most tokens
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return (u ** 6 * rows).to(torch.int32).clamp_(max=rows - 1)


def want_lookup(ids, weight, scale, skip=None):
    import torch
    ids, w = ids.reshape(-1).cpu().long(), weight.double().cpu()
    ok = (ids >= 0) & (ids < len(w))
    if skip is not None:
        ok &= ids != skip
    return torch.where(ok[:, None], w[torch.where(ok, ids, 0)] * scale, 0.0)


def want_grad(ids, grad, rows, scale, skip=None):
    """(gradient, the bound of its 32-bit computation)"""
    import torch
    ids, g = ids.reshape(-1).cpu().long(), grad.double().cpu().reshape(ids.numel(), grad.shape[-1])
    ok = (ids >= 0) & (ids < rows)
    if skip is not None:
        ok &= ids != skip
    total = torch.zeros(rows, g.shape[1], dtype=torch.float64).index_add_(0, ids[ok], g[ok])
    mags = torch.zeros_like(total).index_add_(0, ids[ok], g[ok].abs())
    m = torch.zeros(rows, dtype=torch.float64).index_add_(0, ids[ok], torch.ones(int(ok.sum()), dtype=torch.float64))
    return total * scale, (m[:, None] + 2) * EPS * mags * abs(scale)


@pytest.mark.parametrize("weight,out", [("f32", "f32"), ("f32", "bf16"), ("f32", "f16"), ("f16", "f16"),
                                        ("f16", "f32"), ("f16", "bf16"), ("bf16", "bf16"), ("bf16", "f32"),
                                        ("bf16", "f16")])
@pytest.mark.parametrize("n,rows,dim", [(1, 1, 1), (1, 300, 2048), (7, 5, 7), (33, 257, 1000), (1000, 70_001, 64),
                                        (300, 900, 513), (4099, 768, 136)])
def test_lookup(tok, weight, out, n, rows, dim):
    w, ids, scale = rand((rows, dim), weight, 1), make_ids(n, rows, "uniform"), 1.7
    got = tok.embed(ids, w, scale=scale, dtype=dtypes()[out])
    import numpy as np
    want = want_lookup(ids, w, float(np.float32(scale)))
    assert_close(got, want, EPS * want.abs(), "lookup")


@pytest.mark.parametrize("weight", ["f32", "f16", "bf16"])
def test_lookup_by_one_copies_bits(tok, weight):
    import torch
    w, ids = rand((100, 96), weight, 2), make_ids(500, 100, "skewed")
    w[3, 5], w[4, 6], w[5, 7] = float("inf"), float("-inf"), float("nan")
    got = tok.embed(ids, w)
    assert torch.equal(got.nan_to_num(7.5), w[ids.long()].nan_to_num(7.5))


def test_lookup_of_nothing(tok):
    import torch
    w = rand((10, 16), "f32", 3)
    assert tok.embed(torch.zeros(0, dtype=torch.int32, device="cuda"), w).shape == (0, 16)
    assert tok.embed(make_ids(5, 10, "uniform"), w[:, :0]).shape == (5, 0)
    ids = make_ids(12, 10, "uniform").reshape(3, 4)
    assert torch.equal(tok.embed(ids, w), w[ids.long()])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,first,stride", [(64, 0, 64), (64, 1, 67), (64, 8, 80), (100, 4, 108), (33, 0, 40),
                                              (1, 0, 3)])
def test_strides_and_alignment(tok, dtype, dim, first, stride):
    import torch
    rows, n = 50, 77
    base = rand((rows * stride + first + dim,), dtype, 4)
    w = torch.as_strided(base, (rows, dim), (stride, 1), first)
    ids = make_ids(n, rows, "uniform")
    out_base = torch.full((n * (stride + 3) + 5,), -3.0, dtype=w.dtype, device="cuda")
    out = torch.as_strided(out_base, (n, dim), (stride + 3, 1), 1)
    assert torch.equal(tok.embed(ids, w, out=out), w[ids.long()])
    rest = torch.ones_like(out_base, dtype=torch.bool)
    torch.as_strided(rest, (n, dim), (stride + 3, 1), 1).fill_(False)
    assert bool((out_base[rest] == -3.0).all())
    # a table whose columns are apart, and one row for every id
    assert torch.equal(tok.embed(ids, w.t().contiguous().t()), w[ids.long()])
    assert torch.equal(tok.embed(ids, w[:1].expand(rows, dim)), w[:1].expand(n, dim))


def test_rows_past_2_to_the_31_elements(tok):
    import torch
    rows, dim = 300_000, 8192  # 2.46e9 elements
    w = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([0, 299_999, 262_144, 262_143, 299_999], dtype=torch.int32, device="cuda")
    w[ids.long()] = rand((5, dim), "bf16", 5)
    assert torch.equal(tok.embed(ids, w), w[ids.long()])
    g = rand((5, dim), "bf16", 6)
    w[299_998], w[1] = 1.0, 1.0
    out = tok.embed_grad(ids, g, rows, out=w)
    assert torch.equal(out[262_144], g[2]) and torch.equal(out[0], g[0])
    want = (g[1].float() + g[4].float()).to(torch.bfloat16)
    assert torch.equal(out[299_999], want)
    assert not bool(out[299_998].any()) and not bool(out[1].any())
    assert float(out.abs().amax(dim=1).gt(0).sum()) == 4


def test_ids_out_of_range_and_skipped(bpe, tok):
    import torch
    w = rand((40, 72), "f32", 7) + 10
    ids = make_ids(100, 40, "uniform")
    ids[3], ids[50] = 7, 7
    got = tok.embed(ids, w, skip_id=7)
    assert_close(got, want_lookup(ids, w, 1.0, 7), 0.0, "skipped")
    assert not bool(got[3].any())
    bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)
    pad = ids.clone()
    pad[5] = -1
    got = tok.embed(pad, w, skip_id=-1)
    assert not bool(got[5].any())
    bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)  # a skipped id is no error
    for bad in (40, -2, 2 ** 31 - 1, -2 ** 31 + 1):
        ids[9] = bad
        for call in (lambda: tok.embed(ids, w), lambda: tok.embed_grad(ids, torch.ones(100, 72, device="cuda"), 40)):
            got = call()
            with pytest.raises(bpe.BpeError) as e:
                bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)
            assert e.value.code == 7
            bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)  # cleared
            want = want_lookup(ids, w, 1.0) if got.shape[0] == 100 else \
                want_grad(ids, torch.ones(100, 72), 40, 1.0)[0]
            assert torch.equal(got.double().cpu(), want)
    none = tok.embed(make_ids(4, 5, "uniform"), w[:0])  # no rows: every id is out of range
    assert not bool(none.any())
    with pytest.raises(bpe.BpeError):
        bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("grad,weight", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"),
                                         ("f16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("n,rows,dim,kind", [
    (0, 9, 8, "uniform"), (1, 1, 1, "one"), (1, 1000, 256, "one"), (40, 7, 5, "uniform"), (300, 768, 512, "skewed"),
    (1024, 1025, 33, "down"), (5000, 300, 130, "one"), (5000, 40_000, 72, "skewed"), (20_001, 3000, 24, "skewed"),
    (64, 3, 4104, "uniform"), (129, 2, 16, "down")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient(tok, grad, weight, n, rows, dim, kind, accumulate):
    import torch
    ids, g, scale = make_ids(n, rows, kind), rand((n, dim), grad, 8), 0.375
    old = rand((rows, dim), weight, 9)
    want, bound = want_grad(ids, g, rows, scale)
    if accumulate:
        want = want + old.double().cpu()
        bound = bound + EPS * (want.abs() + bound)
    out = tok.embed_grad(ids, g, rows, scale=scale, out=old.clone(), accumulate=accumulate)
    assert_close(out, want, bound, "gradient")
    again = tok.embed_grad(ids, g, rows, scale=scale, out=old.clone(), accumulate=accumulate)
    assert torch.equal(out, again)  # the order of the sums is fixed
    if accumulate:
        met = torch.zeros(rows, dtype=torch.bool)
        met[ids.long().cpu()] = True
        assert torch.equal(out[~met.cuda()], old[~met.cuda()])


@pytest.mark.parametrize("n", [70_001, 300_003])
def test_gradient_of_many_tokens(tok, n):
    ids, g = make_ids(n, 5000, "skewed"), rand((n, 16), "f32", 10)
    want, bound = want_grad(ids, g, 5000, 1.0)
    assert_close(tok.embed_grad(ids, g, 5000), want, bound, "many tokens")


@pytest.mark.parametrize("grad,weight,dim", [("bf16", "bf16", 1024), ("f32", "f32", 513)])
def test_gradient_of_a_large_table(tok, grad, weight, dim):
    """Many tokens and a table of 80 MB: its zeros are written beside the sums."""
    import torch
    n, rows = 15_000, 40_000
    ids, g = make_ids(n, rows, "skewed"), rand((n, dim), grad, 30)
    want, bound = want_grad(ids, g, rows, 0.5)
    out = torch.full((rows, dim), 3.0, dtype=dtypes()[weight], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            tok.embed_grad(ids, g, rows, scale=0.5, out=out)
        after = out.clone()  # ordered behind the call on its stream
    torch.cuda.current_stream().wait_stream(side)
    assert_close(after, want, bound, "large table")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        tok.embed_grad(ids, g, rows, scale=0.5, out=out)
    out.fill_(5.0)
    graph.replay()
    assert torch.equal(out, after)


@pytest.mark.parametrize("n", [0, 1, 5])
def test_gradient_of_few_tokens_in_more_than_2_to_the_23_rows(tok, n):
    import torch
    rows = 2 ** 23 + 3
    ids = torch.tensor([rows - 1, 0, 7, 0, rows - 1][:n], dtype=torch.int32, device="cuda")
    grad = torch.arange(1, 2 * n + 1, dtype=torch.float32, device="cuda").reshape(n, 2)
    want = torch.zeros(rows, 2, device="cuda").index_add_(0, ids.long(), grad)  # whole numbers: exact in any order
    out = torch.full((rows, 2), 5.0, device="cuda")
    assert torch.equal(tok.embed_grad(ids, grad, rows, out=out), want)
    assert torch.equal(tok.embed_grad(ids, grad, rows, out=out, accumulate=True), 2 * want)


def test_gradient_skips(tok):
    import torch
    ids, g = make_ids(700, 20, "uniform"), rand((700, 40), "f32", 11)
    ids[::3] = -1
    g[::3] = float("nan")  # what is skipped reaches no row
    want, bound = want_grad(torch.where(ids < 0, 99, ids), g, 20, 2.0, 99)
    assert_close(tok.embed_grad(ids, g, 20, scale=2.0, skip_id=-1), want, bound, "skipped")
    assert not bool(tok.embed_grad(torch.full_like(ids, 3), g, 20, skip_id=3).any())


def test_gradient_of_infinities(tok):
    import torch
    ids, g = make_ids(64, 4, "down"), rand((64, 8), "f32", 12)
    g[0, 1], g[1, 2], g[5, 2], g[2, 3] = float("inf"), float("inf"), float("-inf"), float("nan")
    want, bound = want_grad(ids, g, 4, 1.0)
    assert_close(tok.embed_grad(ids, g, 4), want, bound.nan_to_num(0.0, 0.0), "infinities")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,first,stride", [(64, 1, 67), (64, 8, 72), (33, 0, 40), (1, 0, 2)])
def test_gradient_strides(tok, dtype, dim, first, stride):
    import torch
    n, rows = 500, 60
    g = torch.as_strided(rand((n * stride + first + dim,), dtype, 13), (n, dim), (stride, 1), first)
    ids = make_ids(n, rows, "skewed")
    base = torch.full((rows * (stride + 1) + 2,), -3.0, device="cuda")
    out = torch.as_strided(base, (rows, dim), (stride + 1, 1), 1)
    want, bound = want_grad(ids, g, rows, 1.0)
    assert_close(tok.embed_grad(ids, g, rows, out=out), want, bound, "strides")
    rest = torch.ones_like(base, dtype=torch.bool)
    torch.as_strided(rest, (rows, dim), (stride + 1, 1), 1).fill_(False)
    assert bool((base[rest] == -3.0).all())
    # a gradient that is one row for every token, and one with its columns apart
    for x in (g[:1].expand(n, dim), g.t().contiguous().t()):
        want, bound = want_grad(ids, x, rows, 1.0)
        assert_close(tok.embed_grad(ids, x, rows, dtype=torch.float32), want, bound, "broadcast")


def test_gradient_against_differences(tok):
    """The lookup is linear in the table, and with these values every product
    and sum is exact in 32 bits, so differences equal the gradient exactly."""
    import torch
    rows, dim, n, scale, h = 6, 5, 23, 0.5, 0.25
    ids = make_ids(n, rows, "skewed")
    g = torch.Generator(device="cuda")
    g.manual_seed(14)
    w = torch.randint(-8, 9, (rows, dim), generator=g, device="cuda").float()
    c = torch.randint(-8, 9, (n, dim), generator=g, device="cuda").float()
    got = tok.embed_grad(ids, c, rows, scale=scale)
    for r in range(rows):
        for k in range(dim):
            e = torch.zeros_like(w)
            e[r, k] = h
            up = (tok.embed(ids, w + e, scale=scale).double() * c.double()).sum()
            down = (tok.embed(ids, w - e, scale=scale).double() * c.double()).sum()
            assert float((up - down) / (2 * h)) == float(got[r, k])


def test_autograd(tok):
    import torch
    w = rand((30, 24), "f32", 15).requires_grad_()
    ids = make_ids(90, 30, "skewed").reshape(9, 10)
    c = rand((9, 10, 24), "f32", 16)
    (tok.embed(ids, w, scale=3.0) * c).sum().backward()
    want, bound = want_grad(ids, c, 30, 3.0)
    assert_close(w.grad, want, bound, "backward")
    w.grad = None
    tok.embed(ids, w, skip_id=2).sum().backward()  # an upstream gradient that is one broadcast number
    want, bound = want_grad(ids, torch.ones(9, 10, 24), 30, 1.0, 2)
    assert_close(w.grad, want, bound, "broadcast backward")
    with torch.no_grad():
        assert not tok.embed(ids, w).requires_grad


def test_other_streams(bpe, tok):
    import torch
    s = torch.cuda.Stream()
    ids, w, g = make_ids(3000, 500, "skewed"), rand((500, 128), "f32", 17), rand((3000, 128), "f32", 18)
    want = (tok.embed(ids, w), tok.embed_grad(ids, g, 500))
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = (tok.embed(ids, w), tok.embed_grad(ids, g, 500))
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_graph_capture(tok):
    import torch
    ids, w, g = make_ids(2000, 400, "skewed"), rand((400, 72), "bf16", 19), rand((2000, 72), "bf16", 20)
    out, dw = tok.embed(ids, w), tok.embed_grad(ids, g, 400)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        tok.embed(ids, w, out=out)
        tok.embed_grad(ids, g, 400, out=dw)
    ids.copy_(make_ids(2000, 400, "uniform", 5))
    graph.replay()
    assert torch.equal(out, w[ids.long()])
    want, bound = want_grad(ids, g, 400, 1.0)
    assert_close(dw, want, bound, "replayed")


def test_refusals(bpe, tok):
    import torch
    ids, w, out = make_ids(8, 10, "uniform"), rand((10, 16), "f32", 21), torch.zeros(8, 16, device="cuda")
    L = bpe.lib()
    st = torch.cuda.current_stream().cuda_stream
    good = [tok.handle, ids.data_ptr(), 8, w.data_ptr(), 0, 10, 16, 16, 1.0, bpe.NO_ID, out.data_ptr(), 0, 16, st]
    assert L.bpe_embed(*good) == 0
    for at, value in ((0, None), (1, None), (1, ids.data_ptr() + 2), (2, -1), (2, 2 ** 31), (3, None),
                      (3, w.data_ptr() + 2), (4, 3), (4, -1), (5, -1), (5, 2 ** 31), (6, -1), (7, -16), (10, None),
                      (10, out.data_ptr() + 1), (11, 9), (12, 15), (12, -1)):
        assert L.bpe_embed(*(good[:at] + [value] + good[at + 1:])) == 1, (at, value)
        assert b"bpe_embed" in L.bpe_last_error()
    good = [tok.handle, ids.data_ptr(), 8, out.data_ptr(), 0, 16, 1.0, bpe.NO_ID, 10, 16, w.data_ptr(), 0, 16, 0, st]
    assert L.bpe_embed_grad(*good) == 0
    for at, value in ((0, None), (1, None), (2, -1), (2, 2 ** 31), (3, None), (3, out.data_ptr() + 3), (4, 7),
                      (5, -1), (8, -1), (8, 2 ** 31), (9, -1), (10, None), (10, w.data_ptr() + 2), (11, -4),
                      (12, 15), (12, -16)):
        assert L.bpe_embed_grad(*(good[:at] + [value] + good[at + 1:])) == 1, (at, value)
        assert b"bpe_embed_grad" in L.bpe_last_error()
    with pytest.raises(ValueError):
        tok.embed(ids.long(), w)
    with pytest.raises(ValueError):
        tok.embed(ids, w.double())
    with pytest.raises(ValueError):
        tok.embed(ids.cpu(), w)
    with pytest.raises(ValueError):
        tok.embed(ids, w.reshape(-1))
    with pytest.raises(ValueError):
        tok.embed(ids, w, dtype=torch.float64)
    with pytest.raises(ValueError):
        tok.embed(ids, w, out=torch.zeros(8, 15, device="cuda"))
    with pytest.raises(ValueError):
        tok.embed_grad(ids, out[:7], 10)
    with pytest.raises(ValueError):
        tok.embed_grad(ids, out, 10, accumulate=True)
    with pytest.raises(ValueError):
        tok.embed_grad(ids, out, 11, out=torch.zeros(10, 16, device="cuda"))
