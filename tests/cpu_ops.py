"""A Tokenizer whose library calls are done on the host, by numpy on the
addresses that the binding passes: for tests of what the binding itself does."""
from __future__ import annotations

import ctypes

import numpy as np


def _array(address, ctype, count):
    return np.ctypeslib.as_array((ctype * max(count, 1)).from_address(address))[:count] if count else np.zeros(0, ctype)


class Library:
    """bpe_embed, bpe_embed_grad and bpe_adjust_logits of float32 rows without gaps; `calls` names those made."""

    def __init__(self):
        self.calls = []

    def bpe_embed(self, handle, ids, n, weight, weight_type, rows, dim, stride, scale, skip, out, out_type, out_stride,
                  stream):
        self.calls.append("embed")
        assert (weight_type, out_type, stride, out_stride) == (0, 0, dim, dim)
        i = _array(ids, ctypes.c_int32, n)
        ok = (i >= 0) & (i < rows) & (i != skip)
        w = _array(weight, ctypes.c_float, rows * dim).reshape(rows, dim)
        _array(out, ctypes.c_float, n * dim).reshape(n, dim)[:] = np.where(ok[:, None], w[np.where(ok, i, 0)] * scale, 0)
        return 0

    def bpe_embed_grad(self, handle, ids, n, grad, grad_type, stride, scale, skip, rows, dim, out, out_type, out_stride,
                       accumulate, stream):
        self.calls.append("embed_grad")
        assert (grad_type, out_type, stride, out_stride) == (0, 0, dim, dim)
        i = _array(ids, ctypes.c_int32, n)
        ok = (i >= 0) & (i < rows) & (i != skip)
        o = _array(out, ctypes.c_float, rows * dim).reshape(rows, dim)
        if not accumulate:
            o[:] = 0
        np.add.at(o, i[ok], _array(grad, ctypes.c_float, n * dim).reshape(n, dim)[ok] * scale)
        return 0

    def bpe_adjust_logits(self, handle, packed, stream):
        """Halves every logit: enough to see that it was called."""
        import byte_level_bpe_pretokenize_gb300 as bpe
        self.calls.append("adjust_logits")
        self.logits_args = bpe.LogitsArgs.from_buffer_copy(packed)
        a = self.logits_args
        assert a.logits_type == a.out_type == 0
        count = a.n_rows * a.n_vocab
        if count:
            _array(a.out, ctypes.c_float, count)[:] = _array(a.logits, ctypes.c_float, count) * 0.5
        return 0


def tokenizer(monkeypatch):
    """A Tokenizer on the host: torch's CPU tensors have device number -1."""
    import byte_level_bpe_pretokenize_gb300 as bpe
    bpe._torch()
    monkeypatch.setattr(bpe, "_raw_stream", lambda device: 0)
    tok = object.__new__(bpe.Tokenizer)
    tok.device, tok.handle, tok._lib = -1, None, Library()
    return tok
