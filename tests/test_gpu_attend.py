"""Attention over a cache in 4 bits against sums in 64 bits, on caches of random
bytes: types, head layouts, lengths, masks, strides and what is refused."""
import numpy as np
import pytest

from tests import paged_util as pu
from tests.ops_util import assert_close, byte_tokenizer, load

pytestmark = pytest.mark.gpu

PARTS = {"float32": 2, "float16": 1, "bfloat16": 1}


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
    bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)


class Batch:
    """Requests over a random cache: lens tokens each, the last new[r] of them new."""

    def __init__(self, lens, heads, group, dim, block, dtype="bfloat16", new=None, pad=0, seed=0, spare=2, by=1.5):
        import torch
        rng = np.random.default_rng(seed)
        self.lens, self.block, self.dim = np.asarray(lens), block, dim
        self.new = np.ones(len(lens), np.int64) if new is None else np.asarray(new)
        held = -(-self.lens // block)
        blocks = int(held.sum()) + spare
        self.cache = pu.random_cache(rng, blocks, heads, block, dim)
        self.table = np.full((len(lens), max(1, int(held.max(initial=0))) + 1), -1, np.int32)
        order = rng.permutation(blocks)
        for r, h in enumerate(held):
            self.table[r, :h], order = order[:h], order[h:]
        self.unused = order
        self.offsets = None if new is None else np.concatenate([[0], np.cumsum(self.new)])
        tokens = int(self.new.sum()) + pad
        self.q = torch.from_numpy(rng.standard_normal((tokens, heads * group, dim)) * by).to(getattr(torch, dtype))

    def run(self, tok, **k):
        import torch
        k.setdefault("offsets", None if self.offsets is None else torch.from_numpy(self.offsets).cuda())
        return tok.attend(self.q.cuda(), torch.from_numpy(self.cache).cuda(), torch.from_numpy(self.table).cuda(),
                          torch.from_numpy(self.lens.astype(np.int32)).cuda(), self.block, **k)

    def check(self, got, scale=None, label=""):
        import torch
        name = str(self.q.dtype).replace("torch.", "")
        want, bound = pu.attention(self.q.double().numpy(), self.cache, self.table, self.lens, self.block, self.offsets,
                                   scale, PARTS[name])
        none = np.isnan(want).all((1, 2))  # tokens of no request
        if self.offsets is not None:
            none = np.arange(len(want)) >= self.offsets[-1]
        assert not bool(got[torch.from_numpy(none).cuda()].any())
        assert_close(got[torch.from_numpy(~none).cuda()], torch.from_numpy(want[~none]), torch.from_numpy(bound[~none]),
                     label)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("dim", [1, 8, 21, 32, 40, 64, 72, 96, 128, 130, 160, 192, 200, 256])
def test_dims_and_types(tok, dim, dtype):
    b = Batch([1, 33, 70], 2, 3, dim, 16, dtype, seed=dim)
    b.check(b.run(tok))


@pytest.mark.parametrize("dtype,out", [("float32", "bfloat16"), ("bfloat16", "float32"), ("float16", "bfloat16"),
                                       ("bfloat16", "float16")])
def test_result_types(tok, dtype, out):
    import torch
    b = Batch([50, 3], 1, 4, 64, 16, dtype)
    got = b.run(tok, dtype=getattr(torch, out))
    assert got.dtype is getattr(torch, out)
    b.check(got)


@pytest.mark.parametrize("heads,group", [(1, 1), (3, 2), (2, 5), (1, 8), (2, 9), (1, 16), (1, 17), (5, 1), (1, 40)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_head_layouts(tok, heads, group, dtype):
    b = Batch([37, 1, 64, 5], heads, group, 64, 8, dtype, seed=group)
    b.check(b.run(tok))


@pytest.mark.parametrize("block", [1, 2, 3, 7, 16, 31, 32, 33, 100, 256])
def test_blocks(tok, block):
    b = Batch([0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 200], 1, 2, 128, block, seed=block)
    b.check(b.run(tok))


@pytest.mark.parametrize("lens", [[1], [5000], [20_000], [0], [0, 0, 0], [1, 4000, 2, 3, 900], [100] * 300,
                                  list(range(1, 200))])
def test_lengths(tok, lens):
    b = Batch(lens, 2, 2, 32, 16, seed=len(lens))
    b.check(b.run(tok))


def test_many_requests(tok):
    """More than a thread of a block adds up at once; most have no new tokens."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 40, 3000)
    new = np.where(rng.random(3000) < 0.3, rng.integers(0, 4, 3000), 0)
    b = Batch(np.maximum(lens, new), 1, 2, 32, 16, new=new, seed=3)
    b.check(b.run(tok))


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("heads,group,dim", [(2, 4, 64), (1, 1, 128), (2, 3, 40), (1, 16, 256)])
def test_new_tokens_see_those_before_them(tok, heads, group, dim, dtype):
    new = [1, 0, 5, 33, 2, 70, 0]
    b = Batch([40, 9, 5, 64, 200, 70, 0], heads, group, dim, 16, dtype, new=new, pad=4, seed=group)
    b.check(b.run(tok))


# Long runs have kernels of their own where all heads' columns are 8192 at least: 638 tokens of 16 query heads are
# 10,208; with a quarter of the heads the same runs take the others.
@pytest.mark.parametrize("share", [1, 4])
@pytest.mark.parametrize("dtype,heads,group,dim,block", [
    ("bfloat16", 16, 1, 128, 16), ("float16", 4, 4, 64, 16), ("bfloat16", 8, 2, 21, 3), ("float16", 8, 3, 96, 100),
    ("bfloat16", 4, 5, 200, 16), ("float16", 16, 1, 256, 7), ("bfloat16", 4, 8, 32, 1), ("bfloat16", 8, 2, 130, 32)])
def test_long_runs_of_new_tokens(tok, dtype, heads, group, dim, block, share):
    """Runs on either side of a block's columns and of 128 tokens, behind nothing, little and much."""
    new = [128, 1, 300, 64, 129, 0, 16]
    heads = -(-heads // share)
    b = Batch([128, 500, 300, 700, 131, 9, 400], heads, group, dim, block, dtype, new=new, pad=3, seed=dim)
    got = b.run(tok)
    b.check(got)
    assert bool((got == b.run(tok)).all())


@pytest.mark.parametrize("dtype,dim,block", [("bfloat16", 128, 16), ("float16", 64, 5), ("bfloat16", 21, 16),
                                             ("float16", 96, 32)])
def test_long_runs_of_many_heads(tok, dtype, dim, block):
    """Enough columns (322 x 8 of 16 heads) for blocks of two tiles of 128 to keep the GPU busy."""
    new = [128, 1, 129, 64]
    b = Batch([300, 500, 129, 64], 16, 8, dim, block, dtype, new=new, pad=2, seed=dim)
    b.check(b.run(tok))


@pytest.mark.parametrize("scale", [1.0, 0.0, -0.4, 0.01])
def test_long_runs_scale(tok, scale):
    b = Batch([200, 330], 16, 1, 64, 16, new=[200, 330], seed=21)
    b.check(b.run(tok, scale=scale), scale)


def test_long_runs_with_sharp_scores(tok):
    """Scores hundreds apart: results are scaled as the maximum grows."""
    b = Batch([600, 200], 16, 1, 64, 16, "float16", new=[330, 190], seed=22, by=40.0)
    b.check(b.run(tok))


def test_long_runs_that_see_little(tok):
    """Requests that were not served, or only in part: tokens that see nothing get zeros."""
    b = Batch([0, 100, 300, 0], 16, 1, 32, 16, new=[128, 250, 64, 130], seed=23)
    got = b.run(tok)
    b.check(got)
    assert not bool(got[:128 + 150].any()) and bool(got[128 + 150].any())


def test_long_runs_of_strided_queries_and_results(tok):
    import torch
    heads, dim = 16, 64
    b = Batch([300, 260], heads, 1, dim, 16, new=[300, 230], seed=24)
    want = b.run(tok)
    q = b.q
    for start in (0, 1, 4):  # aligned and not
        wide = torch.zeros(530, (heads + 2) * dim + 3, dtype=q.dtype)
        b.q = wide[:, start:start + heads * dim].unflatten(1, (heads, dim))
        b.q.copy_(q)
        out = torch.full((530, (heads + 2) * dim + 3), 7.0, dtype=q.dtype, device="cuda")
        y = out[:, start:start + heads * dim].unflatten(1, (heads, dim))
        given = wide.cuda()[:, start:start + heads * dim].unflatten(1, (heads, dim))
        got = tok.attend(given, torch.from_numpy(b.cache).cuda(), torch.from_numpy(b.table).cuda(),
                         torch.from_numpy(b.lens.astype(np.int32)).cuda(), 16, offsets=torch.from_numpy(b.offsets).cuda(),
                         out=y)
        assert got is y and torch.equal(y, want)
        out[:, start:start + heads * dim] = 7.0
        assert bool((out == 7.0).all())
    b.q = q
    assert b.run(tok, dtype=torch.float32).dtype is torch.float32
    b.check(b.run(tok, dtype=torch.float32))


def test_long_runs_with_values_far_apart(tok):
    """What halves do not hold in one unit is computed in 32 bits: tokens of sizes 2^40 apart, seen by some."""
    b = Batch([400, 300], 12, 2, 64, 16, new=[150, 200], seed=3)
    for r, t, exponent in ((0, 399, 40), (0, 380, -40), (1, 150, 60), (1, 299, 30)):
        page = b.cache[b.table[r, t // 16]]
        at = 16 * 32 + t % 16 * 8
        for which in (0, 1):
            pairs = page[which, 5, at:at + 8].view("<u4")
            for j in range(2):
                step = pu.bf16_value(pairs[j] & 0xFFFF) * np.float32(2.0) ** exponent
                base = pu.bf16_value(pairs[j] >> 16) * np.float32(2.0) ** exponent
                if which == 0:  # keys stay small, so that weights are no ones and zeros
                    step, base = step * np.float32(2.0) ** -exponent, base * np.float32(2.0) ** -exponent
                pairs[j] = pu.bf16_bits(step) | pu.bf16_bits(base) << np.uint32(16)
    b.check(b.run(tok))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_long_runs_do_not_see_nans_that_come_later(tok, dtype):
    b = Batch([300, 260], 13, 2, 64, 16, dtype, new=[200, 130], seed=5)
    want = b.run(tok)
    page = b.cache[b.table[0, 250 // 16]]
    at = 16 * 32 + 250 % 16 * 8
    page[..., at:at + 8] = np.array([0x7FC00000] * 2, "<u4").view(np.uint8)
    got = b.run(tok)
    # new token i sees 100 + i + 1; in 32 bits what comes before may round otherwise
    clean = Batch([300, 260], 13, 2, 64, 16, dtype, new=[200, 130], seed=5)
    assert bool(got[150:200].isnan().all()) and not bool(got[:150].isnan().any())
    got[150:200] = want[150:200]
    clean.check(got)


def test_long_and_short_runs_together(tok):
    """Decode steps among chunks of prompts: each as if alone."""
    import torch
    new = [1, 200, 1, 1, 40, 2, 129, 1]
    lens = [900, 200, 1, 333, 500, 2, 700, 64]
    b = Batch(lens, 6, 4, 128, 16, new=new, seed=12)
    got = b.run(tok)
    b.check(got)
    for r in range(len(new)):
        one = Batch(lens, 6, 4, 128, 16, new=new, seed=12)
        rows = slice(one.offsets[r], one.offsets[r + 1])
        one.q, one.lens, one.table = one.q[rows], one.lens[r:r + 1], one.table[r:r + 1]
        one.new, one.offsets = one.new[r:r + 1], np.array([0, new[r]])
        # the steps are cut elsewhere, so that sums are joined in another order
        one.check(got[rows])
        one.check(one.run(tok))


def test_a_captured_step_with_long_runs(tok):
    import torch
    b = Batch([300, 500, 40], 13, 2, 64, 16, new=[200, 130, 1], seed=8)
    q, cache = b.q.cuda(), torch.from_numpy(b.cache).cuda()
    table, off = torch.from_numpy(b.table).cuda(), torch.from_numpy(b.offsets).cuda()
    lens = torch.from_numpy(b.lens.astype(np.int32)).cuda()
    out = torch.empty_like(q)
    want = tok.attend(q, cache, table, lens, 16, offsets=off)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tok.attend(q, cache, table, lens, 16, offsets=off, out=out)
    for _ in range(2):
        out.fill_(3.0)
        graph.replay()
        assert torch.equal(out, want)


def test_tokens_that_see_nothing(tok):
    """Requests that were not served: fewer tokens in the cache than new ones."""
    b = Batch([0, 3, 0, 10], 2, 2, 64, 16, new=[2, 7, 1, 1], seed=1)
    got = b.run(tok)
    b.check(got)
    assert not bool(got[:2].any()) and not bool(got[2:6].any()) and bool(got[6].any())


def test_scale(tok):
    for scale in (1.0, 0.0, -0.3, 0.01):
        b = Batch([90, 40], 1, 3, 64, 16, "float32", seed=7)
        b.check(b.run(tok, scale=scale), scale)


def test_sharp_scores(tok):
    """Scores hundreds apart, the largest met late: what came before is scaled away."""
    b = Batch([3000, 200], 1, 2, 64, 16, "float32", seed=11, by=40.0)
    b.check(b.run(tok))


@pytest.mark.parametrize("new", [None, [3, 2, 40]])
def test_what_is_not_seen_may_be_anything(tok, new):
    """NaNs and infinities behind a request's end, in blocks of nobody and in tokens that come later."""
    lens = [20, 37, 64]
    clean = Batch(lens, 2, 2, 64, 16, new=new, seed=5)
    want = clean.run(tok)
    dirty = Batch(lens, 2, 2, 64, 16, new=new, seed=5)
    for pairs in (0x7FC00000, 0x7F807F80, 0xFF80FF80, 0xFFFFFFFF):
        for r, length in enumerate(lens):
            for t in range(length, -(-length // 16) * 16):
                page = dirty.cache[dirty.table[r, t // 16]]
                at = 16 * 32 + t % 16 * 8
                page[..., at:at + 8] = np.array([pairs, pairs], "<u4").view(np.uint8)
        for b in dirty.unused:
            dirty.cache[b] = 0xFF
        assert np.array_equal(want.float().cpu().numpy(), dirty.run(tok).float().cpu().numpy())
    if new is None:
        return
    # the last new token of the last request: only its own row may see it
    page = dirty.cache[dirty.table[2, 63 // 16]]
    page[..., 16 * 32 + 15 * 8:16 * 32 + 16 * 8] = np.array([0x7FC00000] * 2, "<u4").view(np.uint8)
    got = dirty.run(tok)
    assert bool(got[-1].isnan().all())
    # with a token that a long run may not read as halves its request is computed by other kernels, whose roundings
    # are others: both are within the bound of the 64-bit result, neither is the other's
    assert np.array_equal(got[:5].float().cpu().numpy(), want[:5].float().cpu().numpy())
    got[-1] = want[-1]
    clean.check(got)


def test_a_nan_is_seen(tok):
    """In one head's values: that head's elements of the group; in its keys: the whole row."""
    b = Batch([50, 50], 2, 2, 64, 16, seed=2)
    want = b.run(tok)
    page = b.cache[b.table[0, 1]]
    nan = np.array([0x7FC00000], "<u4").view(np.uint8)
    page[1, 1, 16 * 32 + 3 * 8 + 4:16 * 32 + 3 * 8 + 8] = nan
    got = b.run(tok)
    assert bool(got[0, 2:, 32:].isnan().all())
    got[0, 2:, 32:] = want[0, 2:, 32:]
    assert bool((got == want).all())
    page[0, 0, 16 * 32:16 * 32 + 4] = nan
    got = b.run(tok)
    assert bool(got[0, :2].isnan().all()) and not bool(got[1].isnan().any())


@pytest.mark.parametrize("lens,new", [([64, 50], None), ([64, 50], [3, 40]), ([300, 290], [300, 200])])
def test_an_infinity_is_seen_by_its_group_alone(tok, lens, new):
    """A base of infinity, which no write leaves, among the values that every token sees."""
    import torch
    heads = 16 if new and new[0] > 200 else 2
    b = Batch(lens, heads, 2, 64, 16, new=new, seed=2)
    clean = Batch(lens, heads, 2, 64, 16, new=new, seed=2)
    page = b.cache[b.table[0, 0]]
    page[1, 1, 16 * 32 + 4:16 * 32 + 8] = np.array([0x7F803E80], "<u4").view(np.uint8)  # token 0, group 1
    got, want = b.run(tok), clean.run(tok)
    rows = slice(0, 1 if new is None else new[0])
    assert not bool(got[rows, 2:4, 32:].isfinite().any())
    got[rows, 2:4, 32:] = want[rows, 2:4, 32:]
    clean.check(got)


def test_strides(tok):
    import torch
    heads, group, dim, block = 2, 3, 64, 16
    b = Batch([40, 90, 7], heads, group, dim, block, seed=9)
    want = b.run(tok)
    q, cache = b.q.cuda(), torch.from_numpy(b.cache).cuda()
    table, lens = torch.from_numpy(b.table).cuda(), torch.from_numpy(b.lens.astype(np.int32)).cuda()
    wide = torch.zeros(3, 10 * dim + 3, dtype=q.dtype, device="cuda")
    layers = torch.randint(0, 256, (cache.shape[0], 3, *cache.shape[1:]), dtype=torch.uint8, device="cuda")
    layers[:, 1] = cache
    tables = torch.full((3, table.shape[1] + 5), 10 ** 6, dtype=torch.int32, device="cuda")
    tables[:, :table.shape[1]] = table
    for start in (0, 1, 4):  # aligned and not
        x = wide[:, start:start + 6 * dim].unflatten(1, (6, dim))
        x.copy_(q)
        out = torch.full((3, 10 * dim + 3), 7.0, dtype=q.dtype, device="cuda")
        y = out[:, start:start + 6 * dim].unflatten(1, (6, dim))
        assert tok.attend(x, layers[:, 1], tables[:, :table.shape[1]], lens, block, out=y) is y
        assert torch.equal(y, want)
        out[:, start:start + 6 * dim] = 7.0
        assert bool((out == 7.0).all())
    t = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(tok.attend(t, cache, table, lens, block), want)
    spread = torch.empty(3, 6, 2 * dim, dtype=q.dtype, device="cuda")
    spread[..., ::2] = q
    assert torch.equal(tok.attend(spread[..., ::2], cache, table, lens, block), want)
    one = q[:1].expand(3, 6, dim)
    assert torch.equal(tok.attend(one, cache, table, lens, block), tok.attend(one.contiguous(), cache, table, lens, block))


def test_rows_of_no_request(tok):
    """Zeros in a new tensor, and left alone in the caller's."""
    import torch
    b = Batch([30, 12], 1, 2, 32, 16, new=[2, 1], pad=5, seed=1)
    got = b.run(tok)
    assert not bool(got[3:].any())
    out = torch.full_like(got, 9.0)
    assert torch.equal(b.run(tok, out=out)[:3], got[:3]) and bool((out[3:] == 9.0).all())
    b.offsets = None
    one = b.run(tok)
    assert not bool(one[2:].any()) and bool(one[:2].any())


def test_equal_inputs_give_equal_bits(tok):
    import torch
    b = Batch([5000, 3, 777], 2, 4, 128, 16, seed=4)
    first = b.run(tok)
    for _ in range(3):
        assert torch.equal(b.run(tok), first)


def test_bad_lengths_and_tables(bpe, tok):
    import torch
    status(bpe, tok)
    b = Batch([40, 50, 60, 70], 1, 2, 64, 16, seed=6)
    want = b.run(tok)
    status(bpe, tok)
    for bad in (-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        b.lens = np.array([40, bad, 60, 70])
        got = b.run(tok)
        with pytest.raises(bpe.BpeError) as e:
            status(bpe, tok)
        assert e.value.code == 7 and not bool(got[1].any()) and torch.equal(got[[0, 2, 3]], want[[0, 2, 3]])
    # a block outside of the cache: its 16 tokens are not seen
    b.lens = np.array([40, 50, 60, 70])
    for bad in (-1, len(b.cache), 2 ** 31 - 1, -2 ** 31):
        kept = b.table[2, 1]
        b.table[2, 1] = bad
        got = b.run(tok)
        with pytest.raises(bpe.BpeError):
            status(bpe, tok)
        b.table[2, 1] = kept
        assert torch.equal(got[[0, 1, 3]], want[[0, 1, 3]])
        cut = Batch([40, 50, 60, 70], 1, 2, 64, 16, seed=6)
        cut.table[2, 1:3] = cut.table[2, 2:4]
        cut.lens[2] = 44
        cut.check(got)
    # no blocks at all
    got = tok.attend(b.q.cuda(), torch.zeros(0, *b.cache.shape[1:], dtype=torch.uint8, device="cuda"),
                     torch.zeros(4, 6, dtype=torch.int32, device="cuda"), torch.full((4,), 9, dtype=torch.int32, device="cuda"), 16)
    with pytest.raises(bpe.BpeError):
        status(bpe, tok)
    assert not bool(got.any())


def test_bad_offsets(bpe, tok):
    import torch
    b = Batch([40, 50, 60], 1, 2, 64, 16, new=[2, 3, 1], seed=6)
    want = b.run(tok)
    status(bpe, tok)
    for offsets, good in (([0, 2, 5, 7], [0, 1, 2, 3, 4]), ([-1, 2, 5, 6], [2, 3, 4, 5]),
                          ([0, 2, 2 ** 40, 6], [0, 1]), ([0, 9, 5, 6], [5])):
        b.offsets = np.array(offsets)
        got = b.run(tok)
        with pytest.raises(bpe.BpeError):
            status(bpe, tok)
        rest = [i for i in range(6) if i not in good]
        assert torch.equal(got[good], want[good]) and not bool(got[rest].any())


def test_empty(tok):
    import torch
    cache = tok.new_cache(2, 16, 1, 32)
    table, lens = torch.zeros(0, 3, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    assert tok.attend(torch.zeros(0, 2, 32, device="cuda"), cache, table, lens, 16).shape == (0, 2, 32)
    assert not bool(tok.attend(torch.ones(3, 2, 32, device="cuda"), cache, table, lens, 16).any())
    table, lens = torch.zeros(3, 0, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    assert not bool(tok.attend(torch.ones(3, 2, 32, device="cuda"), cache, table, lens, 16).any())
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    assert tok.attend(torch.zeros(0, 2, 32, device="cuda"), cache, table, lens, 16, offsets=off).shape == (0, 2, 32)


def test_a_cache_past_4_gigabytes(tok):
    import torch
    heads, dim, block = 8, 128, 256
    b = Batch([700, 300], heads, 2, dim, block, seed=8)
    page = pu.page_bytes(block, dim)
    blocks = 6 * 2 ** 30 // (2 * heads * page)
    cache = torch.empty(blocks, 2, heads, page, dtype=torch.uint8, device="cuda")
    table = np.where(b.table >= 0, b.table * 31 % 97 + blocks - 97, -1).astype(np.int32)
    for i, j in zip(b.table.ravel(), table.ravel()):
        if i >= 0:
            cache[j] = torch.from_numpy(b.cache[i]).cuda()
    got = tok.attend(b.q.cuda(), cache, torch.from_numpy(table).cuda(), torch.from_numpy(b.lens.astype(np.int32)).cuda(),
                     block)
    assert torch.equal(got, b.run(tok))


@pytest.mark.parametrize("new", [None, [300, 290]])
def test_blocks_far_apart(tok, new):
    """Two blocks 33 gigabytes apart: addresses that 32 bits do not hold even in units of 16 bytes."""
    import torch
    heads, dim, block = 16, 32, 512
    b = Batch([400, 300], heads, 1, dim, block, new=new, spare=0, seed=8)
    apart = 33 * 2 ** 30
    try:
        room = torch.empty(apart + b.cache[0].size, dtype=torch.uint8, device="cuda")
    except torch.cuda.OutOfMemoryError:
        pytest.skip("no 33 gigabytes free")
    page = b.cache.shape[-1]
    cache = room.as_strided(b.cache.shape, (apart, heads * page, page, 1))
    cache.copy_(torch.from_numpy(b.cache))
    k = {} if new is None else {"offsets": torch.from_numpy(b.offsets).cuda()}
    got = tok.attend(b.q.cuda(), cache, torch.from_numpy(b.table).cuda(), torch.from_numpy(b.lens.astype(np.int32)).cuda(),
                     block, **k)
    assert torch.equal(got, b.run(tok))
    b.check(got)


def test_replays_follow_lengths_tables_and_queries(tok):
    """A captured decode step, replayed while its inputs change in place."""
    import torch
    b = Batch([900, 40], 2, 4, 128, 16, seed=3)
    q, cache = b.q.cuda(), torch.from_numpy(b.cache).cuda()
    table = torch.zeros(2, 80, dtype=torch.int32, device="cuda")
    table[:, :b.table.shape[1]] = torch.from_numpy(b.table).cuda()
    lens = torch.from_numpy(b.lens.astype(np.int32)).cuda()
    tok.attend(q, cache, table, lens, 16)
    graphs, outs = [], []
    for _ in range(2):  # two graphs share the workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(tok.attend(q, cache, table, lens, 16))
        graphs.append(graph)
    for a, c in ((900, 40), (17, 0), (1, 40), (512, 39)):
        lens.copy_(torch.tensor([a, c]))
        q.copy_(torch.randn_like(q))
        want = tok.attend(q, cache, table, lens, 16)
        for graph, out in zip(graphs, outs):
            out.fill_(5.0)
            graph.replay()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_on_another_stream(tok):
    import torch
    b = Batch([2000, 40], 2, 4, 64, 16, seed=3)
    want = b.run(tok)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = b.run(tok)
    side.synchronize()
    assert torch.equal(got, want)


def test_no_derivative(tok):
    import torch
    b = Batch([20, 3], 1, 2, 32, 16, "float32")
    want = b.run(tok)
    b.q.requires_grad_()
    got = b.run(tok)
    assert torch.equal(got, want)
    with pytest.raises(RuntimeError, match="no gradient"):
        got.sum().backward()
    with pytest.raises(ValueError):
        b.run(tok, out=torch.empty_like(want))


def test_refusals(bpe, tok):
    import torch
    b = Batch([20, 3], 2, 2, 32, 16)
    q, cache = b.q.cuda(), torch.from_numpy(b.cache).cuda()
    table, lens = torch.from_numpy(b.table).cuda(), torch.from_numpy(b.lens.astype(np.int32)).cuda()
    for bad in (lambda: tok.attend(q.double(), cache, table, lens, 16), lambda: tok.attend(q[0], cache, table, lens, 16),
                lambda: tok.attend(q[:, :3], cache, table, lens, 16), lambda: tok.attend(q, cache, table, lens, 8),
                lambda: tok.attend(q, cache, table, lens.long(), 16), lambda: tok.attend(q, cache, table.long(), lens, 16),
                lambda: tok.attend(q, cache, table, lens[:1], 16), lambda: tok.attend(q, cache, table[0], lens, 16),
                lambda: tok.attend(q, cache, table, lens, 16, offsets=lens.long()),
                lambda: tok.attend(q, cache.cpu(), table, lens, 16),
                lambda: tok.attend(q, cache, table, lens, 16, dtype=torch.float64),
                lambda: tok.attend(q, cache, table, lens, 16, out=torch.empty(2, 4, 31, device="cuda")),
                lambda: tok.attend(q[:, :0], cache, table, lens, 16)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(bpe.BpeError, match="below one new token"):
        tok.attend(q[:1], cache, table, lens, 16)
    with pytest.raises(bpe.BpeError, match="scale"):
        tok.attend(q, cache, table, lens, 16, scale=float("nan"))
    with pytest.raises(bpe.BpeError, match="overlap"):
        tok.attend(q, cache, table, lens, 16, out=torch.empty(1, 4, 32, dtype=q.dtype, device="cuda").expand(2, 4, 32))
