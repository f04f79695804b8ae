"""Results that would overlap what they are computed from are refused by the
library before it touches the GPU: attend, and rotate but for a whole tensor in
place. Rows side by side in one tensor are not. (Calls that are not refused end
here with another error, as there is no GPU or no handle behind the pointer.)"""
import ctypes
import itertools

import numpy as np
import pytest


@pytest.fixture(scope="module")
def bpe():
    import __graft_entry__
    __graft_entry__.build()
    import byte_level_bpe_pretokenize_gb300 as m
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers here are no device pointers")
    return m


HANDLE = ctypes.create_string_buffer(1 << 16)  # not null; zeros
BASE = 1 << 20


def refused(bpe, call, word):
    with pytest.raises(bpe.BpeError) as e:
        call()
    return e.value.code == 1 and word in str(e.value)


def attend(bpe, q, out, tokens, rows, dim, q_type=2, out_type=2):
    """q and out: (byte offset, token stride, head stride)."""
    size = {0: 4, 1: 2, 2: 2}
    a = bpe.AttendArgs(queries=BASE + q[0], out=BASE + out[0], query_type=q_type, out_type=out_type,
                       query_token_stride=q[1], query_head_stride=q[2], out_token_stride=out[1], out_head_stride=out[2],
                       n_tokens=tokens, n_heads=1, group=rows, dim=dim, cache=BASE, n_blocks=1, block_stride=1 << 20,
                       block_size=16, table=BASE, max_blocks=1, table_stride=1, seq_lens=BASE, offsets=None,
                       n_requests=1, scale=1.0)
    assert size[q_type]
    return refused(bpe, lambda: bpe.bpe_attend(ctypes.addressof(HANDLE), a, 0), "out overlaps queries")


def rotate(bpe, x, out, tokens, heads, dim, x_type=2, out_type=2):
    return refused(bpe, lambda: bpe.bpe_rotate(ctypes.addressof(HANDLE), BASE + x[0], x_type, tokens, heads, dim, x[1],
                                               x[2], BASE, BASE, dim // 2, False, False, 1.0, BASE + out[0], out_type,
                                               out[1], out[2], 0), "out overlaps x")


def test_what_overlaps(bpe):
    whole = (0, 4 * 64, 64)
    n = 10 * 4 * 64 * 2  # bytes of 10 tokens of 4 x 64 in 16 bits
    assert attend(bpe, whole, whole, 10, 4, 64)
    assert not rotate(bpe, whole, whole, 10, 4, 64)  # in place
    for call in (attend, rotate):
        for at in (2, 128, 512, n - 2):
            assert call(bpe, whole, (at, 256, 64), 10, 4, 64) and call(bpe, (at, 256, 64), whole, 10, 4, 64)
        for at in (n, n + 2, 10 * n):
            assert not call(bpe, whole, (at, 256, 64), 10, 4, 64) and not call(bpe, (at, 256, 64), whole, 10, 4, 64)
        # 32-bit results of 16-bit rows
        assert call(bpe, (n, 256, 64), (0, 256, 64), 10, 4, 64, out_type=0)
        assert not call(bpe, (2 * n, 256, 64), (0, 256, 64), 10, 4, 64, out_type=0)
        # other strides: heads before tokens, a result among wider rows
        assert call(bpe, whole, (64, 64, 640), 10, 4, 64)
        assert call(bpe, whole, (n - 256, 2000, 64), 10, 4, 64)
        assert not call(bpe, whole, (n, 2000, 64), 10, 4, 64)
        # one token, one head
        assert call(bpe, (0, 0, 64), (64, 0, 64), 1, 4, 64) and not call(bpe, (0, 0, 64), (512, 0, 64), 1, 4, 64)
        assert call(bpe, (0, 64, 0), (64, 64, 0), 10, 1, 64) and not call(bpe, (0, 64, 0), (1280, 64, 0), 10, 1, 64)


def test_rows_side_by_side(bpe):
    for call in (attend, rotate):
        # parts of a fused row of 12 heads: heads 0..3 and 4..7, either way, and heads 3..6
        assert not call(bpe, (0, 768, 64), (512, 768, 64), 10, 4, 64)
        assert not call(bpe, (512, 768, 64), (0, 768, 64), 10, 4, 64)
        assert call(bpe, (0, 768, 64), (384, 768, 64), 10, 4, 64)
        # halves of each head, every other token
        assert not call(bpe, (0, 512, 128), (128, 512, 128), 10, 4, 64)
        assert call(bpe, (0, 512, 128), (126, 512, 128), 10, 4, 64)
        assert not call(bpe, (0, 512, 64), (512, 512, 64), 10, 4, 64)
        # one row of queries for all tokens and heads
        assert not call(bpe, (0, 0, 0), (128, 256, 64), 10, 4, 64)
        assert call(bpe, (128 + 512, 0, 0), (128, 256, 64), 10, 4, 64)


def test_against_every_byte(bpe):
    """Equal strides: exactly where two rows share a byte, of all small layouts."""
    rng = np.random.default_rng(0)
    seen = set()
    for _ in range(3000):
        n, m, dim = rng.integers(1, 5, 3)
        # rows of one tensor must not meet among themselves
        t = dim + rng.integers(0, 8)
        s = (m - 1) * t + dim + rng.integers(0, 3 * t)
        if rng.random() < 0.3:
            s, t = dim + rng.integers(0, 4), 0
            t = (n - 1) * s + dim + rng.integers(0, 9)
        at = int(rng.integers(0, 2 * (n * s + m * t))) if rng.random() < 0.9 else int(rng.integers(0, 4))
        x = {2 * (i * s + j * t + k) for i, j, k in itertools.product(range(n), range(m), range(dim))}
        y = {2 * at + b for b in x}
        if at == 0:
            continue
        got = rotate(bpe, (0, int(s), int(t)), (2 * at, int(s), int(t)), int(n), int(m), int(dim))
        assert got == bool(x & y), (n, m, dim, s, t, at)
        seen.add(got)
    assert seen == {True, False}
