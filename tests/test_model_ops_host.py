"""Host side of the operators around the model (no GPU): null handles, the
argument structure's layout, and the constants of the header."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def bpe():
    import __graft_entry__
    __graft_entry__.build()
    import byte_level_bpe_pretokenize_gb300 as m
    return m


@pytest.fixture(scope="module")
def header():
    return open(os.path.join(ROOT, "include", "bpe_gb300.h")).read()


def test_null_handles(bpe):
    L = bpe.lib()
    assert L.bpe_embed(None, None, 0, None, 0, 0, 0, 0, 1.0, 0, None, 0, 0, None) == 1
    assert b"bpe_embed: null handle" in L.bpe_last_error()
    assert L.bpe_embed_grad(None, None, 0, None, 0, 0, 1.0, 0, 0, 0, None, 0, 0, 0, None) == 1
    assert L.bpe_plan_blocks(None, None, None, 0, 16, None, 0, None, None, 0, 0, None, None, None, 0, None, None) == 1
    assert L.bpe_adjust_logits(None, ctypes.byref(bpe.LogitsArgs()), None) == 1
    assert b"bpe_adjust_logits: null handle" in L.bpe_last_error()


def test_type_codes(bpe, header):
    for name, value in (("BPE_F32", bpe.F32), ("BPE_F16", bpe.F16), ("BPE_BF16", bpe.BF16)):
        assert f"#define {name} {value}\n" in header


def test_logits_args_are_the_headers(bpe, header):
    body = re.search(r"typedef struct bpe_logits_args \{(.*?)\} bpe_logits_args;", header, re.S).group(1)
    kinds = {"const void*": ctypes.c_void_p, "void*": ctypes.c_void_p, "int": ctypes.c_int, "int64_t": ctypes.c_int64}
    fields = []
    for line in body.strip().split(";"):
        if not line.strip():
            continue
        kind, names = re.match(r"\s*((?:const )?\w+\*?)\s+(.*)", line.strip()).groups()
        kind = kinds.get(kind, ctypes.c_void_p if kind.endswith("*") else None)
        fields += [(n.strip(), kind) for n in names.split(",")]
    assert fields == bpe.LogitsArgs._fields_


def test_packed_arguments_are_the_structure(bpe):
    values = list(range(1, len(bpe.LogitsArgs._fields_) + 1))
    raw = bpe._pack_logits(*values)
    assert len(raw) == ctypes.sizeof(bpe.LogitsArgs)
    args = bpe.LogitsArgs.from_buffer_copy(raw)
    assert [getattr(args, n) for n, _ in args._fields_] == values
