"""The embedding gradient on either side of every choice between its kernels:
the single launch (up to 512 tokens), places by rank (up to 12,288), sorts of
one, two and three passes by one CTA or a cluster, tokens held in registers or
read again, zeros beside the sums. Upstream gradients are small whole numbers,
so that sums are exact in any order."""
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


def check(bpe, tok, n, rows, dim, dtype="float32", skip=None, bad=False):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(n + dim)
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    ids = (u ** 4 * rows).long().clamp_(max=rows - 1)
    ids[:2], ids[-2:] = rows - 1, 0  # the ends of the table, first and last
    ids = ids.to(torch.int32)
    if skip is not None:
        ids[n // 3:n // 2] = skip
    if bad:
        ids[n // 2:n // 2 + 9:2] = rows
        ids[n // 2 + 1:n // 2 + 9:2] = -5
    grad = torch.randint(-4, 5, (n, dim), generator=g, device="cuda").to(getattr(torch, dtype))
    ok = (ids >= 0) & (ids < rows)
    if skip is not None:
        ok &= ids != skip
    want = torch.zeros(rows, dim, device="cuda").index_add_(0, ids[ok].long(), grad[ok].float())
    out = torch.full((rows, dim), 3.0, device="cuda")
    got = tok.embed_grad(ids, grad, rows, scale=0.5, skip_id=skip, out=out)
    assert torch.equal(got, want * 0.5)
    tok.embed_grad(ids, grad, rows, scale=0.25, skip_id=skip, out=out, accumulate=True)
    assert torch.equal(out, want * 0.75)
    try:
        bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)
        reported = 0
    except bpe.BpeError as e:
        reported = e.code
    assert reported == (7 if bad else 0)


@pytest.mark.parametrize("n", [511, 512, 513, 1023, 12_287, 12_288, 12_289, 12_320])
@pytest.mark.parametrize("rows,dim", [(3000, 64), (3000, 77), (50_000, 8), (1, 5)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_edges(bpe, tok, n, rows, dim, dtype):
    check(bpe, tok, n, rows, dim, dtype)


@pytest.mark.parametrize("n", [20_000, 65_536, 65_537, 70_001])
@pytest.mark.parametrize("rows,dim", [(1, 9), (700, 24), (1023, 5), (1024, 8), (2 ** 20 - 1, 3), (2 ** 20, 3),
                                      (2 ** 20 + 5, 3), (2 ** 20 + 5, 20)])
def test_passes(bpe, tok, n, rows, dim):
    """One, two and three passes; 20 columns of 2^20 rows are 84 MB, whose zeros have a stream of their own."""
    check(bpe, tok, n, rows, dim)


@pytest.mark.parametrize("n", [513, 600, 1024, 2047, 2048, 2049, 12_289])
@pytest.mark.parametrize("dim", [2, 5])
def test_few_tokens_of_a_table_too_large_to_rank(bpe, tok, n, dim):
    check(bpe, tok, n, 2 ** 23 + 3, dim)


@pytest.mark.parametrize("n,rows", [(300, 900), (5000, 900), (20_000, 900), (20_000, 40_000), (70_001, 2 ** 20 + 5),
                                    (1500, 2 ** 23 + 3)])
def test_skipped_and_wrong_ids(bpe, tok, n, rows):
    check(bpe, tok, n, rows, 6, skip=7)
    check(bpe, tok, n, rows, 8, "float16", skip=-1, bad=True)


@pytest.mark.parametrize("n", [1_000_003, 4_000_001])
def test_millions_of_tokens(bpe, tok, n):
    check(bpe, tok, n, 32_256, 4)
