"""Block tables, cache slots and positions against plain Python integers (every
value has to be equal)."""
import random

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


def plain(offsets, cached, table, free, block, n_slots, head):
    n = len(table)
    table = [list(r) for r in table]
    if offsets is None:
        offsets = list(range(n + 1))
    cached = cached or [0] * n
    room, given, taken = len(free) - head, 0, 0
    slots, positions, seq = [-1] * n_slots, [0] * n_slots, []
    for i in range(n):
        c, m = cached[i], offsets[i + 1] - offsets[i]
        held, want = -(-c // block), -(-(c + m) // block)
        gets = want - held
        given += gets
        served = gets == 0 or given <= room
        if given <= room:
            taken = given
        if served:
            table[i][held:want] = free[head + given - gets:head + given]
        seq.append(c + m if served else c)
        for t in range(offsets[i], offsets[i + 1]):
            p = c + t - offsets[i]
            positions[t] = p
            if served:
                slots[t] = table[i][p // block] * block + p % block
    return table, seq, slots, positions, [head + taken, max(0, given - room)]


def run(tok, offsets, cached, table, free, block, n_slots=None, head=None, width=None):
    import torch

    def dev(x, dtype):
        return None if x is None else torch.tensor(x, dtype=dtype, device="cuda")

    t = dev(table, torch.int32).reshape(len(table), -1)
    if width:  # rows further apart than their entries
        wide = torch.full((len(table), width), -9, dtype=torch.int32, device="cuda")
        wide[:, :t.shape[1]] = t
        t = wide[:, :t.shape[1]]
    got = tok.plan_blocks(dev(offsets, torch.int64), dev(cached, torch.int32), t, dev(free, torch.int32), block,
                          n_slots=n_slots, head=dev(None if head is None else [head], torch.int64))
    if width:
        assert bool((wide[:, t.shape[1]:] == -9).all())
    return [t.tolist()] + [g.tolist() for g in got]


def make(rng, n, block, longest, cached_most, single=False):
    cached = [rng.choice([0, rng.randint(0, cached_most), block * rng.randint(0, cached_most // block)])
              for _ in range(n)]
    lens = [1] * n if single else [rng.choice([0, 1, rng.randint(0, longest)]) for _ in range(n)]
    offsets = [0]
    for m in lens:
        offsets.append(offsets[-1] + m)
    most = max([-(-(c + m) // block) for c, m in zip(cached, lens)] + [1])
    pool = list(range(n * most + sum(-(-(c + m) // block) + 1 for c, m in zip(cached, lens)) + 7))
    rng.shuffle(pool)
    table = [[pool.pop() if k < -(-c // block) else -1 for k in range(most)] for c in cached]
    return cached, offsets, table, pool


@pytest.mark.parametrize("n,block,longest,cached_most", [
    (1, 16, 1, 0), (1, 1, 40, 9), (2, 7, 30, 100), (5, 256, 3000, 700), (33, 32, 100, 1000), (300, 16, 60, 500),
    (1024, 8, 30, 100), (1025, 3, 9, 40), (2500, 100, 300, 20), (9000, 16, 12, 64)])
@pytest.mark.parametrize("share", [1.0, 0.5, 0.0])
def test_requests(tok, n, block, longest, cached_most, share):
    rng = random.Random(n * 1000 + block)
    cached, offsets, table, free = make(rng, n, block, longest, cached_most)
    need = sum(-(-(c + b - a) // block) - -(-c // block) for c, a, b in zip(cached, offsets, offsets[1:]))
    head = rng.randint(0, 3)
    free = free[:head + int(need * share)]
    n_slots = offsets[-1] + rng.choice([0, 1, 130])
    want = plain(offsets, cached, table, free, block, n_slots, head)
    assert run(tok, offsets, cached, table, free, block, n_slots, head) == list(want)
    assert run(tok, offsets, cached, table, free, block, n_slots, head, width=len(table[0]) + 5) == list(want)


@pytest.mark.parametrize("n,block,cached_most", [(1, 16, 0), (7, 16, 5000), (256, 1, 30), (3000, 64, 2000)])
@pytest.mark.parametrize("share", [1.0, 0.4])
def test_single_tokens(tok, n, block, cached_most, share):
    rng = random.Random(n + block)
    cached, _, table, free = make(rng, n, block, 1, cached_most, single=True)
    need = sum(-(-(c + 1) // block) - -(-c // block) for c in cached)
    free = free[:int(need * share)]
    assert run(tok, None, cached, table, free, block) == list(plain(None, cached, table, free, block, n, 0))
    want = plain(None, cached, table, free, block, n + 9, 0)
    assert run(tok, None, cached, table, free, block, n + 9) == list(want)


@pytest.mark.parametrize("n", [513, 1208, 2048, 2049, 4097])
@pytest.mark.parametrize("block", [1, 16])
def test_single_tokens_of_several_tiles(tok, n, block):
    """One launch up to 2048 requests and two above, with tiles that do not begin at the first request."""
    rng = random.Random(n)
    cached, _, table, free = make(rng, n, block, 1, 40, single=True)
    want = plain(None, cached, table, free, block, n + 77, 1)
    assert run(tok, None, cached, table, free, block, n + 77, 1) == list(want)


def test_prompts_without_a_cache(tok):
    rng = random.Random(5)
    _, offsets, table, free = make(rng, 50, 16, 200, 0)
    want = plain(offsets, None, table, free, 16, offsets[-1], 0)
    assert run(tok, offsets, None, table, free, 16, offsets[-1]) == list(want)


def test_one_long_request_among_empty_ones(tok):
    lens = [0, 0, 70_000, 0, 1, 0]
    offsets = [0]
    for m in lens:
        offsets.append(offsets[-1] + m)
    cached = [0, 16, 33, 5, 0, 0]
    table = [[-1] * 4400 for _ in lens]
    for i, c in enumerate(cached):
        for k in range(-(-c // 16)):
            table[i][k] = 100_000 + 10 * i + k
    free = list(range(4400, 0, -1))
    want = plain(offsets, cached, table, free, 16, offsets[-1] + 3, 0)
    assert run(tok, offsets, cached, table, free, 16, offsets[-1] + 3) == list(want)


@pytest.mark.parametrize("n", [5, 3000])
def test_many_empty_requests_in_a_tile(tok, n):
    """More requests start at one token than a tile has tokens."""
    offsets = [0] * (n // 2) + [7] * (n - n // 2) + [2000]
    cached = [(i * 7) % 40 for i in range(n)]
    table = [[i * 100 + k if k < -(-c // 16) else -1 for k in range(130)] for i, c in enumerate(cached)]
    free = list(range(900_000, 900_400))
    want = plain(offsets, cached, table, free, 16, 2000, 2)
    assert run(tok, offsets, cached, table, free, 16, 2000, 2) == list(want)


def test_no_requests(tok):
    import torch
    table = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    free = torch.arange(5, dtype=torch.int32, device="cuda")
    off = torch.zeros(1, dtype=torch.int64, device="cuda")
    seq, slots, pos, info = tok.plan_blocks(off, None, table, free, 16, n_slots=3)
    assert seq.numel() == 0 and slots.tolist() == [-1] * 3 and pos.tolist() == [0] * 3 and info.tolist() == [0, 0]
    seq, slots, pos, info = tok.plan_blocks(None, None, table, free, 16)
    assert slots.numel() == 0 and info.tolist() == [0, 0]


def test_slots_past_32_bits(tok):
    blocks = [2 ** 31 - 1, 2 ** 31 - 2, 17]
    cached, table, free = [300, 0], [[blocks[0], blocks[2], -1], [-1, -1, -1]], [blocks[1]]
    got = run(tok, None, cached, table, free, 256)
    assert got[2] == [17 * 256 + 44, (2 ** 31 - 2) * 256]
    assert got == list(plain(None, cached, table, free, 256, 2, 0))


def test_the_head_moves_on_the_device(tok):
    """Steps without a host wait: info[0] of a step is the head of the next."""
    import torch
    rng = random.Random(8)
    n, block = 20, 4
    table = torch.full((n, 12), -1, dtype=torch.int32, device="cuda")
    free_list = list(range(100, 200))
    rng.shuffle(free_list)
    free = torch.tensor(free_list, dtype=torch.int32, device="cuda")
    info = torch.zeros(2, dtype=torch.int64, device="cuda")
    cached = torch.zeros(n, dtype=torch.int32, device="cuda")
    plain_table, plain_cached, head = [[-1] * 12 for _ in range(n)], [0] * n, 0
    for _ in range(10):
        cached, _, _, info = tok.plan_blocks(None, cached, table, free, block, head=info[:1])
        plain_table, plain_cached, _, _, (head, lack) = plain(None, plain_cached, plain_table, free_list, block, n, head)
        assert lack == 0
    assert table.tolist() == plain_table and cached.tolist() == plain_cached and info.tolist() == [head, 0]
    used = [b for row in plain_table for b in row if b >= 0]
    assert len(set(used)) == len(used)


def _status(bpe, tok):
    import torch
    try:
        bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)
    except bpe.BpeError as e:
        return e.code
    return 0


def test_bad_lengths_are_left_out(bpe, tok):
    table = [[1, 2, -1], [3, -1, -1], [4, -1, -1], [5, -1, -1]]
    free = [9, 8, 7, 6]
    assert _status(bpe, tok) == 0
    # a negative cached length: that request alone is not served
    got = run(tok, None, [20, -5, 16, 3], table, free, 16)
    assert _status(bpe, tok) == 7 and _status(bpe, tok) == 0
    assert got[1] == [21, 0, 17, 4] and got[2] == [2 * 16 + 4, -1, 9 * 16, 5 * 16 + 3]
    assert got[0] == [[1, 2, -1], [3, -1, -1], [4, 9, -1], [5, -1, -1]] and got[4] == [1, 0]
    # more blocks than a table row holds
    got = run(tok, None, [48, 5, 16, 3], table, free, 16)
    assert _status(bpe, tok) == 7
    assert got[1] == [48, 6, 17, 4] and got[2][0] == -1 and got[0][0] == [1, 2, -1]
    # offsets past the slots, or falling
    got = run(tok, [0, 2, 4, 30, 31], None, table, free, 16, n_slots=8)
    assert _status(bpe, tok) == 7
    assert got[1] == [2, 2, 0, 0] and got[2] == [144, 145, 128, 129, -1, -1, -1, -1]
    run(tok, [0, 5, 3, 6, 8], None, table, free, 16, n_slots=8)
    assert _status(bpe, tok) == 7
    run(tok, [-3, 5, 6, 7, 8], None, table, free, 16, n_slots=8)
    assert _status(bpe, tok) == 7
    # a head outside the free list: no block is left
    for head in (-1, 5):
        got = run(tok, None, [16, 3, 0, 5], table, free, 16, head=head)
        assert _status(bpe, tok) == 7
        assert got[1] == [16, 4, 0, 6] and got[0] == table and got[4][1] == 2


def test_refusals(bpe, tok):
    import torch
    n = 4
    off = torch.arange(n + 1, dtype=torch.int64, device="cuda")
    cached = torch.zeros(n, dtype=torch.int32, device="cuda")
    table = torch.zeros(n, 3, dtype=torch.int32, device="cuda")
    free = torch.arange(9, dtype=torch.int32, device="cuda")
    head = torch.zeros(2, dtype=torch.int64, device="cuda")
    seq, slots, pos, info = tok.plan_blocks(off, cached, table, free, 16, n_slots=n)
    L = bpe.lib()
    good = [tok.handle, off.data_ptr(), cached.data_ptr(), n, 16, free.data_ptr(), 9, head.data_ptr(),
            table.data_ptr(), 3, 3, seq.data_ptr(), slots.data_ptr(), pos.data_ptr(), n, info.data_ptr(),
            torch.cuda.current_stream().cuda_stream]
    assert L.bpe_plan_blocks(*good) == 0
    for at, value in ((0, None), (1, off.data_ptr() + 4), (2, cached.data_ptr() + 1), (3, -1), (3, 2 ** 31), (4, 0),
                      (4, -16), (4, 2 ** 31), (5, None), (5, free.data_ptr() + 2), (6, -1), (7, head.data_ptr() + 4),
                      (8, None), (8, table.data_ptr() + 2), (9, -1), (10, 2), (11, None), (11, seq.data_ptr() + 1),
                      (12, None), (12, slots.data_ptr() + 4), (13, None), (13, pos.data_ptr() + 2), (14, -1),
                      (14, 2 ** 31), (15, None), (15, info.data_ptr() + 4), (15, head.data_ptr()),
                      (7, info.data_ptr() + 8), (11, cached.data_ptr()), (11, cached.data_ptr() + 12)):
        assert L.bpe_plan_blocks(*(good[:at] + [value] + good[at + 1:])) == 1, (at, value)
        assert b"bpe_plan_blocks" in L.bpe_last_error()
    assert L.bpe_plan_blocks(*([tok.handle, None] + good[2:14] + [n - 1] + good[15:])) == 1
    for args in ((off, cached, table, free, 16), (off[:-1], cached, table, free, 16, 4),
                 (off, cached[:3], table, free, 16, 4), (off, cached.long(), table, free, 16, 4),
                 (off.int(), cached, table, free, 16, 4), (off, cached, table.t(), free, 16, 4),
                 (off, cached, table, free[::2], 16, 4), (off.cpu(), cached, table, free, 16, 4)):
        with pytest.raises(ValueError):
            tok.plan_blocks(*args)
    with pytest.raises(bpe.BpeError):
        tok.plan_blocks(off, cached, table, free, 0, n_slots=n)
