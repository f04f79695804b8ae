"""Host side of the operators on a paged cache (no GPU): tables of rotary
positions, sizes of pages, null handles, the argument structure's layout, and
what the binding refuses before the library is called."""
import ctypes
import math
import os
import re
from fractions import Fraction

import numpy as np
import pytest

from tests import paged_util as pu
from tests.cpu_ops import tokenizer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def bpe():
    import __graft_entry__
    __graft_entry__.build()
    import byte_level_bpe_pretokenize_gb300 as m
    return m


class Library:
    """Names the calls that reach the library."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture()
def tok(bpe, monkeypatch):
    t = tokenizer(monkeypatch)
    t._lib = Library()
    return t


def test_null_handles(bpe):
    L = bpe.lib()
    assert L.bpe_rotate(None, None, 0, 0, 0, 0, 0, 0, None, None, 0, 0, 0, 1.0, None, 0, 0, 0, None) == 1
    assert b"bpe_rotate: null handle" in L.bpe_last_error()
    assert L.bpe_cache_write(None, None, 0, None, None, 0, 1, 32, 0, 0, 0, 0, None, 0, 0, 16, None) == 1
    assert b"bpe_cache_write: null handle" in L.bpe_last_error()
    assert L.bpe_cache_read(None, None, 0, None, 0, 0, 16, 1, 32, None, None, 0, 0, 0, 0, 0, None) == 1
    assert L.bpe_attend(None, ctypes.byref(bpe.AttendArgs()), None) == 1
    assert b"bpe_attend: null handle" in L.bpe_last_error()
    assert L.bpe_cache_page_bytes(16, 128, None) == 1


def test_attend_args_are_the_headers(bpe):
    header = open(os.path.join(ROOT, "include", "bpe_gb300.h")).read()
    body = re.search(r"typedef struct bpe_attend_args \{(.*?)\} bpe_attend_args;", header, re.S).group(1)
    kinds = {"int": ctypes.c_int, "int64_t": ctypes.c_int64, "float": ctypes.c_float}
    fields = []
    for line in body.strip().split(";"):
        if line.strip():
            kind, names = re.match(r"\s*((?:const )?\w+\*?)\s+(.*)", line.strip()).groups()
            kind = kinds.get(kind, ctypes.c_void_p if kind.endswith("*") else None)
            fields += [(n.strip(), kind) for n in names.split(",")]
    assert fields == bpe.AttendArgs._fields_
    values = list(range(1, len(fields) + 1))
    raw = bpe._pack_attend(*values)
    assert len(raw) == ctypes.sizeof(bpe.AttendArgs)
    args = bpe.AttendArgs.from_buffer_copy(raw)
    assert [getattr(args, n) for n, _ in args._fields_] == values


def test_page_bytes(bpe):
    for block in (1, 2, 3, 16, 100, 1 << 20):
        for dim in (1, 31, 32, 33, 64, 96, 128, 129, 160, 161, 200, 224, 256):
            assert bpe.bpe_cache_page_bytes(block, dim) == pu.page_bytes(block, dim)
    for block, dim in ((0, 64), (16, 0), (16, 257), ((1 << 20) + 1, 64), (-1, 64), (16, -3)):
        with pytest.raises(bpe.BpeError) as e:
            bpe.bpe_cache_page_bytes(block, dim)
        assert e.value.code == 1


def test_codes_fill_a_row():
    for dim in (1, 32, 64, 72, 96, 128, 160, 200, 256):
        n = pu.groups(dim) * 32
        assert sorted(pu.code_place(e, dim) for e in range(n)) == list(range(n))


PI = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)


def test_rotary_table_of_given_frequencies(bpe):
    f = [1.0, 0.5, 1e-3, 1e-12, 0.0, 6.25, -0.75, -1e-5, 100.0]
    got = bpe.bpe_rotary_table(len(f), frequencies=f)
    for turn, x in zip(got, f):
        exact = Fraction(x) / (2 * PI)
        off = (Fraction(int(turn), 2 ** 64) - exact) % 1
        off = min(off, 1 - off)
        # two roundings of a 64-bit number, the fraction's own unit, and what taking whole turns off rounds
        assert off <= abs(exact) * Fraction(3, 2 ** 53) + Fraction(2, 2 ** 64) + (Fraction(1, 2 ** 53) if x < 0 else 0)


def test_rotary_table_scales(bpe):
    def turns(t):
        return t.astype(np.float64) * 2.0 ** -64

    plain = 10_000.0 ** (-np.arange(32) / 32) / (2 * math.pi)
    near = dict(rtol=1e-14, atol=2.0 ** -64)  # a table holds whole multiples of 2^-64
    np.testing.assert_allclose(turns(bpe.bpe_rotary_table(32)), plain, **near)
    np.testing.assert_allclose(turns(bpe.bpe_rotary_table(32, base=5e5)), 5e5 ** (-np.arange(32) / 32) / (2 * math.pi), **near)
    np.testing.assert_allclose(turns(bpe.bpe_rotary_table(32, factor=8.0)), plain / 8, **near)
    keep = np.clip((4096 * plain - 1) / 31, 0, 1)
    np.testing.assert_allclose(turns(bpe.bpe_rotary_table(32, factor=8.0, original=4096, low=1.0, high=32.0)),
                               plain * (keep + (1 - keep) / 8), **near)
    assert bpe.bpe_rotary_table(0).shape == (0,)


def test_rotary_table_refusals(bpe):
    for k in (dict(base=0.0), dict(base=-1.0), dict(base=math.nan), dict(base=math.inf), dict(factor=0.0),
              dict(factor=math.inf), dict(factor=math.nan), dict(original=-1.0), dict(original=math.nan),
              dict(original=4096, low=4.0, high=4.0), dict(original=4096, low=math.nan),
              dict(frequencies=[1.0, math.nan]), dict(frequencies=[math.inf, 1.0])):
        with pytest.raises(bpe.BpeError) as e:
            bpe.bpe_rotary_table(2, **k)
        assert e.value.code == 1
    with pytest.raises(bpe.BpeError):
        bpe.bpe_rotary_table(-1)
    with pytest.raises(ValueError):
        bpe.bpe_rotary_table(3, frequencies=[1.0])


def test_binding_refusals(tok):
    import torch
    x, p, t = torch.ones(4, 2, 16), torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int64)
    cache, slots = torch.zeros(3, 2, 2, pu.page_bytes(4, 16), dtype=torch.uint8), torch.arange(4)
    table, lens = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    tracked = x.clone().requires_grad_()
    for bad in (lambda: tok.rotate(x.double(), p, t), lambda: tok.rotate(x[0], p, t), lambda: tok.rotate(x, p[1:], t),
                lambda: tok.rotate(x, p.long(), t), lambda: tok.rotate(x, p, t.int()),
                lambda: tok.rotate(x[..., :15], p, t), lambda: tok.rotate(tracked, p, t, out=torch.empty(4, 2, 16)),
                lambda: tok.rotate(x, p, t, out=torch.empty(4, 2, 16).requires_grad_()),
                lambda: tok.rotate(x, p, t, out=torch.empty(4, 16, 2).transpose(1, 2)),
                lambda: tok.write_cache(cache, slots, x, x.half(), 4), lambda: tok.write_cache(cache, slots, x, x, 8),
                lambda: tok.write_cache(cache, slots, tracked, x, 4), lambda: tok.write_cache(cache, slots[:3], x, x, 4),
                lambda: tok.write_cache(cache.int(), slots, x, x, 4),
                lambda: tok.write_cache(cache[:, :1], slots, x, x, 4),
                lambda: tok.write_cache(cache, slots, x[:, :1], x[:, :1], 4),
                lambda: tok.read_cache(cache, slots, 48, 4), lambda: tok.read_cache(cache, slots.int(), 16, 4),
                lambda: tok.read_cache(cache, slots, 16, 4, dtype=torch.int8),
                lambda: tok.attend(x[:, :1], cache, table, lens, 4), lambda: tok.attend(x, cache, table, lens[1:], 4),
                lambda: tok.attend(x, cache, table.t(), lens, 4), lambda: tok.attend(x, cache, table.long(), lens, 4),
                lambda: tok.attend(x, cache, table, lens, 4, offsets=torch.zeros(4, dtype=torch.int64)),
                lambda: tok.attend(tracked, cache, table, lens, 4, out=torch.empty(4, 2, 16)),
                lambda: tok.attend(x, cache, table, lens, 4, out=torch.empty(4, 2, 16), dtype=torch.float16)):
        with pytest.raises(ValueError):
            bad()
    assert not tok._lib.calls
    tok.rotate(x, p, t), tok.write_cache(cache, slots, x, x, 4), tok.read_cache(cache, slots, 16, 4)
    tok.attend(x, cache, table, lens, 4)
    assert tok._lib.calls == ["bpe_rotate", "bpe_cache_write", "bpe_cache_read", "bpe_attend"]


def test_writes_count_as_writes(tok):
    import torch
    x = torch.ones(4, 2, 16)
    cache, out = torch.zeros(3, 2, 2, pu.page_bytes(4, 16), dtype=torch.uint8), torch.empty(4, 2, 16)
    before = cache._version, out._version
    tok.write_cache(cache, torch.arange(4), x, x, 4)
    tok.rotate(x, torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int64), out=out)
    assert cache._version > before[0] and out._version > before[1]
