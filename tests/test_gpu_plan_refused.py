"""Block plans whose offsets fall: requests that begin below an earlier offset
are refused, and what is served is served whole. Against plain Python integers."""
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
    """As bpe_plan_blocks states it: (table, seq_lens, slots, positions, info), and which requests are served."""
    n, width = len(table), len(table[0])
    table = [list(r) for r in table]
    room, given, taken, high = len(free) - head, 0, 0, offsets[0]
    slots, positions, seq, who = [-1] * n_slots, [0] * n_slots, [], []
    for i in range(n):
        c, a, b = cached[i], offsets[i], offsets[i + 1]
        high = max(high, a)
        ok = 0 <= a <= b <= n_slots and a == high and c >= 0 and -(-(c + b - a) // block) <= width
        held = -(-c // block)
        gets = -(-(c + b - a) // block) - held if ok else 0
        given += gets
        served = ok and (gets == 0 or given <= room)
        if given <= room:
            taken = given
        if served:
            table[i][held:held + gets] = free[head + given - gets:head + given]
            who.append(i)
        seq.append(c + b - a if served else max(c, 0))
        if ok:
            for t in range(a, b):
                positions[t] = c + t - a
                slots[t] = table[i][positions[t] // block] * block + positions[t] % block if served else -1
    return [table, seq, slots, positions, [head + taken, max(0, given - room)]], who


def check(bpe, tok, offsets, cached, table, free, block, n_slots, head=0):
    import torch

    def dev(x, dtype):
        return torch.tensor(x, dtype=dtype, device="cuda")

    t = dev(table, torch.int32)
    got = tok.plan_blocks(dev(offsets, torch.int64), dev(cached, torch.int32), t, dev(free, torch.int32), block,
                          n_slots=n_slots, head=dev([head], torch.int64))
    got = [t.tolist()] + [g.tolist() for g in got]
    with pytest.raises(bpe.BpeError) as e:
        bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)
    assert e.value.code == 7
    want, served = plain(offsets, cached, table, free, block, n_slots, head)
    assert got == want
    # no two requests share a token or a block, and every block that one was dealt is in its table
    blocks = [b for i in served for b in want[0][i][:-(-want[1][i] // block)]]
    assert -1 not in blocks and len(set(blocks)) == len(blocks)
    assert sum(s >= 0 for s in want[2]) == sum(offsets[i + 1] - offsets[i] for i in served)


@pytest.mark.parametrize("block", [1, 2, 16])
@pytest.mark.parametrize("offsets", [[0, 5, 3, 6, 8], [4, 0, 3, 6, 8], [0, 8, 0, 8], [0, 2, 100, 3, 6, 7],
                                     [0, 4, 2, 2, 4, 4, 8], [0, 3, 6, 8, 1], [-3, 5, 2, 6],
                                     [0, 2 ** 62, -2 ** 62, 4, 8], [2 ** 63 - 1, -2 ** 63, 0, 8]])
def test_few_requests(bpe, tok, offsets, block):
    n = len(offsets) - 1
    cached = [(3 * i) % 5 for i in range(n)]
    table = [[100 + 10 * i + k if k < -(-c // block) else -1 for k in range(14)] for i, c in enumerate(cached)]
    check(bpe, tok, offsets, cached, table, list(range(50)), block, 8)
    check(bpe, tok, offsets, cached, table, list(range(50)), block, 8, head=46)


@pytest.mark.parametrize("n", [40, 700, 2048, 2049, 5000, 20_000])
@pytest.mark.parametrize("block", [1, 16])
@pytest.mark.parametrize("falls", [1, 7])
@pytest.mark.parametrize("share", [1.0, 0.5])
def test_many_requests(bpe, tok, n, block, falls, share):
    """Offsets that rise but for a few wrong ones: too low, too high, or two that changed places."""
    rng = random.Random(n + block + falls)
    offsets = [0]
    for _ in range(n):
        offsets.append(offsets[-1] + rng.choice([0, 1, 1, rng.randint(0, 9)]))
    n_slots = offsets[-1] + 5
    for _ in range(falls):
        i = rng.randint(1, n - 1)
        kind = rng.randint(0, 2)
        if kind == 0:
            offsets[i] = rng.randint(-3, max(offsets[i] - 1, -2))
        elif kind == 1:
            offsets[i] = min(offsets[i] + rng.randint(1, 40), n_slots)
        else:
            offsets[i], offsets[i + 1] = offsets[i + 1], offsets[i]
    offsets[n // 2] = offsets[n // 2 + 1] + 1  # one falls in any case
    cached = [rng.randint(0, 20) for _ in range(n)]
    width = 70 // block + 3
    free = list(range(n_slots + n))
    rng.shuffle(free)
    free = free[:2 + int(share * n_slots / block)]
    table = [[1_000_000 + 100 * i + k if k < -(-c // block) else -1 for k in range(width)]
             for i, c in enumerate(cached)]
    check(bpe, tok, offsets, cached, table, free, block, n_slots, head=2)
