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


def encode(tok, n):
    import torch
    data = (torch.arange(n, device="cuda") * 7919 % 251).to(torch.uint8)
    ids, offsets = tok.encode(data, torch.tensor([0, n], device="cuda"))
    assert torch.equal(ids, data.to(torch.int32)) and offsets.tolist() == [0, n]


def test_a_graph_outlives_its_workspace(bpe, tok):
    """Calls that need more than a captured one must not free what it uses."""
    import torch
    n, rows, dim = 4864, 900, 512
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    ids = torch.randint(0, rows, (n,), generator=g, device="cuda", dtype=torch.int32)
    grad = torch.randint(-8, 9, (n, dim), generator=g, device="cuda").float()  # sums are exact in any order
    requests = 3000
    cached = torch.full((requests,), 32, dtype=torch.int32, device="cuda")
    table = torch.zeros(requests, 4, dtype=torch.int32, device="cuda")
    free = torch.arange(requests, dtype=torch.int32, device="cuda")

    def calls():
        return tok.embed_grad(ids, grad, rows), tok.plan_blocks(None, cached, table, free, 16)[1]

    want_grad = torch.zeros(rows, dim, device="cuda").index_add_(0, ids.long(), grad)
    calls()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, slots = calls()
    held = bpe.bpe_workspace_bytes(tok.handle)
    encode(tok, 1 << 20)  # 13 bytes of workspace a byte
    grown = bpe.bpe_workspace_bytes(tok.handle)
    assert grown > held + 13 * (1 << 20)  # the captured block is still there
    blocks = [torch.full((held,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]  # would take its place
    for _ in range(2):
        out.fill_(7.0), slots.fill_(-5)
        graph.replay()
        assert torch.equal(out, want_grad)
        assert torch.equal(slots, free.long() * 16)
    assert all(bool((b == 255).all()) for b in blocks)
    encode(tok, 1 << 21)  # no graph holds the block that this one outgrows: 16 bytes a byte, with room to grow
    assert bpe.bpe_workspace_bytes(tok.handle) - held < 18 * (1 << 21)
    out.fill_(7.0)
    graph.replay()
    assert torch.equal(out, want_grad)
