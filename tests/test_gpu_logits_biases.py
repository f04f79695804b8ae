"""A row with far more biases than the rows beside it, many tokens with several:
the same sums, in time that is linear in the biases. Bounds: test_gpu_logits."""
import pytest

from tests.ops_util import assert_close, byte_tokenizer, load
from tests.test_gpu_logits import call, make, plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tok():
    t = byte_tokenizer(load())
    yield t
    t.close()


def heavy(n, vocab, ids, row, dtype="f32", prompt=50, output=20, masks=0):
    """Rows of which `row` alone has biases: those of `ids`."""
    import torch
    s = make(n, vocab, prompt, output, None, masks, vocab, dtype)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    values = torch.randn(ids.numel(), generator=g, device="cuda")
    s["bias"] = (ids, values, torch.where(torch.arange(n + 1, device="cuda") <= row, 0, ids.numel()))
    return s


def ids_of(kind, m, vocab):
    import torch
    k = torch.arange(m, device="cuda")
    if kind == "one each":
        k = k * 7919 % vocab
    elif kind == "pairs":
        k = k // 2 * 7919 % vocab
    elif kind == "one token":
        k = k * 0 + 1234
    elif kind == "few tokens":  # 700 of them, each in places far apart
        k = k % 700 * 13
    elif kind == "mixed":
        k = torch.where(k % 3 == 0, k, k // 40 * 11) % vocab
    return k.to(torch.int32)


@pytest.mark.parametrize("kind", ["one each", "pairs", "one token", "few tokens", "mixed"])
@pytest.mark.parametrize("dtype,masks", [("f32", 0), ("bf16", 3)])
@pytest.mark.parametrize("m,vocab", [(30_000, 113_645), (9000, 32_256)])
def test_heavy_row(tok, kind, dtype, masks, m, vocab):
    import torch
    s = heavy(64, vocab, ids_of(kind, m, vocab), 5, dtype, masks=masks)
    want, bound = plain(s)
    got = call(tok, s)
    assert_close(got, want, bound, kind)
    assert torch.equal(call(tok, s), got)
    assert_close(call(tok, s, out=s["logits"]), want, bound, f"{kind} in place")


def test_time_of_a_heavy_row(tok):
    """30,000 biases, in pairs, against as many for a token each. The pairs walk
    the list once for every 512 of them in a chunk of 16,384 tokens (about five
    times); searching the list for each took hundreds of times as long."""
    import torch
    times = {}
    for kind in ("one each", "pairs"):
        s = heavy(64, 113_645, ids_of(kind, 30_000, 113_645), 5, "bf16")
        out = torch.empty_like(s["logits"])
        for _ in range(3):
            call(tok, s, out=out)
        best = float("inf")
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            call(tok, s, out=out)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        times[kind] = best
    print({k: f"{v * 1e3:.0f} us" for k, v in times.items()})
    assert times["pairs"] < 12 * times["one each"], times
