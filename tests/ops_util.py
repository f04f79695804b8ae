"""Helpers for the tests of the operators around the model: a tokenizer handle
of the 256 bytes, unit roundoffs, and error bounds."""
from __future__ import annotations

import numpy as np

# unit roundoff (half the spacing relative to the value) and half the smallest subnormal
ROUNDOFF = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float32": 2.0 ** -150, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}


def byte_tokenizer(bpe):
    return bpe.Tokenizer(np.zeros((0, 3), np.int32), np.arange(256, dtype=np.uint8), np.arange(257, dtype=np.int64))


def load():
    """The built package, and a skip without a CUDA device."""
    import pytest
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import byte_level_bpe_pretokenize_gb300 as bpe
    return bpe


def type_name(dtype):
    return str(dtype).replace("torch.", "")


def assert_close(got, want, computed, label=""):
    """|got - want| <= computed + the rounding of want to got's type: `computed`
    bounds the error of the 32-bit computation, element by element."""
    import torch
    name = type_name(got.dtype)
    got, want = got.double().cpu(), want.double().cpu()
    computed = torch.as_tensor(computed, dtype=torch.float64).cpu()
    fin = torch.isfinite(want)
    assert torch.equal(fin, torch.isfinite(got)), f"{label}: finite in other places"
    bad = ~fin & ~((got == want) | (got.isnan() & want.isnan()))
    assert not bool(bad.any()), f"{label}: another infinity or NaN"
    bound = computed + ROUNDOFF[name] * (want.abs() + computed) + TINY[name]
    over = fin & ((got - want).abs() > bound)
    if bool(over.any()):
        at = tuple(int(i) for i in over.nonzero()[0])
        raise AssertionError(f"{label}: {int(over.sum())} of {over.numel()} off, first at {at}: got {got[at]}, "
                             f"want {want[at]}, bound {bound.expand_as(want)[at]}")
