"""Python binding of the GB300 batched byte-level BPE encoder.

Argument marshalling only: every step of the encoder runs in the CUDA kernels
of ``libbpe_gb300.so`` behind the C ABI in ``include/bpe_gb300.h``. There is
no CPU fallback; loading fails loudly when the library is missing.

Low level: ``bpe_build``, ``bpe_encode_batch``, ``bpe_encode_batch_noalloc``,
``bpe_pretokenize_batch``, ``bpe_decode_batch``, ``bpe_sync_status``,
``bpe_destroy`` take device pointers as integers, exactly like the C calls;
``bpe_encode_batch_host`` takes host pointers.
High level: ``Tokenizer`` takes torch CUDA tensors and the current stream.
"""
from __future__ import annotations

import ctypes
import os
import struct
import subprocess
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
_CSRC = os.path.join(_HERE, "csrc")
_BUILD = os.path.join(_HERE, "_build")
LIB_PATH = os.path.join(_BUILD, "libbpe_gb300.so")
NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-cudart", "shared"]

BPE_OK = 0
ERRORS = {1: "INVALID_ARG", 2: "CAPACITY", 3: "CUDA", 4: "BAD_TABLE", 5: "TIMEOUT", 6: "INTERNAL", 7: "BAD_INPUT"}


class BpeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"BPE_ERR_{ERRORS.get(code, code)}: {msg}")
        self.code = code


UNITS = ("bpe_kernels.cu", "model_ops.cu")  # translation units, compiled in parallel


def _sources():
    return [os.path.join(_CSRC, f) for f in sorted(os.listdir(_CSRC)) if f.endswith((".cu", ".cuh", ".inc"))] + \
        [os.path.join(_ROOT, "include", "bpe_gb300.h")]


def build(force: bool = False, nvcc: str = "nvcc") -> str:
    """Compile the CUDA library in-tree for sm_103a (cross-compiles without a GPU)."""
    if not force and os.path.exists(LIB_PATH) and \
            all(os.path.getmtime(LIB_PATH) >= os.path.getmtime(s) for s in _sources()):
        return LIB_PATH
    os.makedirs(_BUILD, exist_ok=True)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    objects = [f"{tmp}.{u}.o" for u in UNITS]
    runs = [subprocess.Popen([nvcc, *NVCC_FLAGS, "-c", "-o", o, os.path.join(_CSRC, u)])
            for u, o in zip(UNITS, objects)]
    codes = [r.wait() for r in runs]
    for r, code in zip(runs, codes):
        if code:
            raise subprocess.CalledProcessError(code, r.args)
    subprocess.check_call([nvcc, *NVCC_FLAGS, "-shared", "-o", tmp, *objects])
    for o in objects:
        os.remove(o)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


_lock = threading.Lock()
_lib = None

EXPORTS = ["bpe_build", "bpe_encode_batch", "bpe_encode_batch_host", "bpe_encode_batch_noalloc", "bpe_pretokenize_batch", "bpe_decode_batch", "bpe_set_word_cache",
           "bpe_set_timing_events", "bpe_set_phase_events", "bpe_set_call_memo", "bpe_sync_status", "bpe_table_info", "bpe_table_monotone", "bpe_merges_monotone",
           "bpe_workspace_bytes", "bpe_train", "bpe_plan_blocks", "bpe_embed", "bpe_embed_grad", "bpe_adjust_logits", "bpe_destroy", "bpe_last_error"]


def lib():
    """The loaded C library (raises if it was never built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: run __graft_entry__.build() "
                                   "(the encoder has no CPU fallback)")
            L = ctypes.CDLL(LIB_PATH)
            i64, i32, p = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
            L.bpe_build.restype = ctypes.c_int
            L.bpe_build.argtypes = [p, i64, p, p, i64, ctypes.c_int, ctypes.POINTER(p)]
            L.bpe_encode_batch.restype = ctypes.c_int
            L.bpe_encode_batch.argtypes = [p, p, i64, p, i64, p, i64, p, p, p]
            L.bpe_encode_batch_host.restype = ctypes.c_int
            L.bpe_encode_batch_host.argtypes = [p, p, i64, p, i64, p, i64, p, p, p]
            L.bpe_encode_batch_noalloc.restype = ctypes.c_int
            L.bpe_encode_batch_noalloc.argtypes = [p, p, i64, p, i64, p, i64, p, p, p]
            L.bpe_pretokenize_batch.restype = ctypes.c_int
            L.bpe_pretokenize_batch.argtypes = [p, i64, p, i64, p, p]
            L.bpe_decode_batch.restype = ctypes.c_int
            L.bpe_decode_batch.argtypes = [p, p, i64, p, i64, p, i64, p, p, p]
            L.bpe_set_word_cache.restype = ctypes.c_int
            L.bpe_set_word_cache.argtypes = [p, ctypes.c_int]
            L.bpe_set_timing_events.restype = ctypes.c_int
            L.bpe_set_timing_events.argtypes = [p, p, p]
            L.bpe_set_call_memo.restype = ctypes.c_int
            L.bpe_set_call_memo.argtypes = [p, ctypes.c_int]
            L.bpe_set_phase_events.restype = ctypes.c_int
            L.bpe_set_phase_events.argtypes = [p, p, ctypes.c_int]
            L.bpe_sync_status.restype = ctypes.c_int
            L.bpe_sync_status.argtypes = [p, p]
            L.bpe_table_info.restype = ctypes.c_int
            L.bpe_table_info.argtypes = [p, ctypes.POINTER(i64), ctypes.POINTER(i64)]
            L.bpe_table_monotone.restype = ctypes.c_int
            L.bpe_table_monotone.argtypes = [p, ctypes.POINTER(ctypes.c_int)]
            L.bpe_merges_monotone.restype = ctypes.c_int
            L.bpe_merges_monotone.argtypes = [p, i64, i64, ctypes.POINTER(ctypes.c_int)]
            L.bpe_train.restype = ctypes.c_int
            L.bpe_train.argtypes = [p, p, p, i64, i64, ctypes.c_int, p, ctypes.POINTER(i64)]
            i, f = ctypes.c_int, ctypes.c_float
            L.bpe_embed.restype = ctypes.c_int
            L.bpe_embed.argtypes = [p, p, i64, p, i, i64, i64, i64, f, i32, p, i, i64, p]
            L.bpe_embed_grad.restype = ctypes.c_int
            L.bpe_embed_grad.argtypes = [p, p, i64, p, i, i64, f, i32, i64, i64, p, i, i64, i, p]
            L.bpe_plan_blocks.restype = ctypes.c_int
            L.bpe_plan_blocks.argtypes = [p, p, p, i64, i64, p, i64, p, p, i64, i64, p, p, p, i64, p, p]
            L.bpe_adjust_logits.restype = ctypes.c_int
            L.bpe_adjust_logits.argtypes = [p, p, p]
            L.bpe_workspace_bytes.restype = ctypes.c_int
            L.bpe_workspace_bytes.argtypes = [p, ctypes.POINTER(i64)]
            L.bpe_destroy.restype = ctypes.c_int
            L.bpe_destroy.argtypes = [p]
            L.bpe_last_error.restype = ctypes.c_char_p
            L.bpe_last_error.argtypes = []
            _lib = L
    return _lib


def _check(rc: int) -> None:
    if rc != BPE_OK:
        raise BpeError(rc, lib().bpe_last_error().decode(errors="replace"))


# ------------------------------------------------------------ C-ABI mirror --

def bpe_build(merges, vocab_bytes, vocab_offsets, device: int = 0) -> int:
    """Host arrays in, opaque handle (int) out. See include/bpe_gb300.h."""
    m = np.ascontiguousarray(np.asarray(merges, dtype=np.int32).reshape(-1, 3))
    vb = np.ascontiguousarray(vocab_bytes, dtype=np.uint8)
    vo = np.ascontiguousarray(vocab_offsets, dtype=np.int64)
    h = ctypes.c_void_p()
    _check(lib().bpe_build(m.ctypes.data if m.size else None, len(m), vb.ctypes.data if vb.size else None,
                           vo.ctypes.data, len(vo) - 1, device, ctypes.byref(h)))
    return h.value


def bpe_encode_batch(handle: int, d_bytes: int, n_bytes: int, d_doc_offsets: int, n_docs: int, d_out_ids: int,
                     out_capacity: int, d_out_offsets: int, want_total: bool, stream: int) -> int | None:
    total = ctypes.c_int64(-1)
    _check(lib().bpe_encode_batch(handle, d_bytes, n_bytes, d_doc_offsets, n_docs, d_out_ids, out_capacity,
                                  d_out_offsets, ctypes.byref(total) if want_total else None, stream))
    return total.value if want_total else None


def bpe_encode_batch_host(handle: int, h_bytes: int, n_bytes: int, h_doc_offsets: int, n_docs: int,
                          h_out_ids: int, out_capacity: int, h_out_offsets: int, want_total: bool,
                          stream: int) -> int | None:
    """bpe_encode_batch on host buffers (pointers as integers; page-locked
    for overlap): copies in, encodes and copies out in a pipeline of slices."""
    total = ctypes.c_int64(-1)
    _check(lib().bpe_encode_batch_host(handle, h_bytes, n_bytes, h_doc_offsets, n_docs, h_out_ids, out_capacity,
                                       h_out_offsets, ctypes.byref(total) if want_total else None, stream))
    return total.value if want_total else None


NOALLOC_MAX_BYTES = 4 << 20  # batch limit of bpe_encode_batch_noalloc's fixed scratch


def bpe_encode_batch_noalloc(handle: int, d_bytes: int, n_bytes: int, d_doc_offsets: int, n_docs: int,
                             d_out_ids: int, out_capacity: int, d_out_offsets: int, want_total: bool,
                             stream: int) -> int | None:
    """bpe_encode_batch on fixed static scratch: allocates no device memory,
    n_bytes <= NOALLOC_MAX_BYTES, one call in flight per device."""
    total = ctypes.c_int64(-1)
    _check(lib().bpe_encode_batch_noalloc(handle, d_bytes, n_bytes, d_doc_offsets, n_docs, d_out_ids, out_capacity,
                                          d_out_offsets, ctypes.byref(total) if want_total else None, stream))
    return total.value if want_total else None


def bpe_pretokenize_batch(d_bytes: int, n_bytes: int, d_doc_offsets: int, n_docs: int, d_start_bits: int,
                          stream: int) -> None:
    _check(lib().bpe_pretokenize_batch(d_bytes, n_bytes, d_doc_offsets, n_docs, d_start_bits, stream))


def bpe_decode_batch(handle: int, d_ids: int, n_ids: int, d_id_offsets: int, n_docs: int, d_out_bytes: int,
                     out_capacity: int, d_out_byte_offsets: int, want_total: bool, stream: int) -> int | None:
    total = ctypes.c_int64(-1)
    _check(lib().bpe_decode_batch(handle, d_ids, n_ids, d_id_offsets, n_docs, d_out_bytes, out_capacity,
                                  d_out_byte_offsets, ctypes.byref(total) if want_total else None, stream))
    return total.value if want_total else None


def bpe_set_word_cache(handle: int, enable: bool) -> None:
    _check(lib().bpe_set_word_cache(handle, 1 if enable else 0))


def bpe_train(word_bytes, word_offsets, word_counts, n_merges: int, device: int = 0):
    """Merge rows int32[k, 3] (left, right, new_id) trained on the GPU from a
    word list (host arrays: bytes, offsets[n + 1], counts[n])."""
    wb = np.ascontiguousarray(word_bytes, dtype=np.uint8)
    wo = np.ascontiguousarray(word_offsets, dtype=np.int64)
    wc = np.ascontiguousarray(word_counts, dtype=np.int64)
    out = np.zeros((max(1, n_merges), 3), dtype=np.int32)
    made = ctypes.c_int64(0)
    _check(lib().bpe_train(wb.ctypes.data if wb.size else None, wo.ctypes.data, wc.ctypes.data if wc.size else None,
                           len(wo) - 1, n_merges, device, out.ctypes.data, ctypes.byref(made)))
    return out[:made.value].copy()


MEMO_OFF, MEMO_ON, MEMO_AUTO = 0, 1, 2


def bpe_set_call_memo(handle: int, mode: int) -> None:
    """Per-call memo of word-cache misses: MEMO_OFF, MEMO_ON or MEMO_AUTO (on
    exactly when the word cache is off)."""
    _check(lib().bpe_set_call_memo(handle, mode))


def bpe_set_timing_events(handle: int, ev_start: int | None, ev_stop: int | None) -> None:
    """cudaEvent_t handles (ints) recorded before the first and after the
    last kernel of each encode call."""
    _check(lib().bpe_set_timing_events(handle, ev_start, ev_stop))


ENCODE_LAUNCHES = 9
ENCODE_KERNELS = ("k_prep_docs", "k_prep_long", "k_tiles", "k_misses", "k_giants", "k_scan_tiles",
                  "k_scan_tile_sums", "k_compact", "k_giant_copy")


class PhaseEvents:
    """ENCODE_LAUNCHES + 1 cudaEvent_t handles (ints) held in a C array that
    lives as long as this object; bpe_set_phase_events records them around
    each kernel of the next encode calls."""

    def __init__(self, events: list[int]):
        if len(events) != ENCODE_LAUNCHES + 1:
            raise ValueError(f"need {ENCODE_LAUNCHES + 1} events")
        self.array = (ctypes.c_void_p * len(events))(*events)


def bpe_set_phase_events(handle: int, events: "PhaseEvents | None") -> None:
    if events is None:
        _check(lib().bpe_set_phase_events(handle, None, 0))
    else:
        _check(lib().bpe_set_phase_events(handle, ctypes.cast(events.array, ctypes.c_void_p), len(events.array)))


def bpe_sync_status(handle: int, stream: int) -> None:
    _check(lib().bpe_sync_status(handle, stream))


def bpe_table_info(handle: int) -> tuple[int, int]:
    a, b = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().bpe_table_info(handle, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def bpe_table_monotone(handle: int) -> bool:
    m = ctypes.c_int()
    _check(lib().bpe_table_monotone(handle, ctypes.byref(m)))
    return bool(m.value)


def bpe_merges_monotone(merges, n_vocab: int) -> bool:
    """Host-only: whether every merge's operands are bytes or made by lower ranks."""
    mm = np.ascontiguousarray(np.asarray(merges, dtype=np.int32).reshape(-1, 3))
    out = ctypes.c_int()
    _check(lib().bpe_merges_monotone(mm.ctypes.data if mm.size else None, len(mm), n_vocab, ctypes.byref(out)))
    return bool(out.value)


def bpe_workspace_bytes(handle: int) -> int:
    """Device workspace the handle holds now (0 until a call needs it)."""
    b = ctypes.c_int64()
    _check(lib().bpe_workspace_bytes(handle, ctypes.byref(b)))
    return b.value


F32, F16, BF16 = 0, 1, 2  # element types of the operators below
NO_ID = -2 ** 31  # a skip_id that no token has


def bpe_embed(handle: int, d_ids: int, n_ids: int, d_weight: int, weight_type: int, n_rows: int, dim: int,
              weight_stride: int, scale: float, skip_id: int, d_out: int, out_type: int, out_stride: int,
              stream: int) -> None:
    _check(lib().bpe_embed(handle, d_ids, n_ids, d_weight, weight_type, n_rows, dim, weight_stride, scale, skip_id,
                           d_out, out_type, out_stride, stream))


def bpe_embed_grad(handle: int, d_ids: int, n_ids: int, d_grad_out: int, grad_out_type: int, grad_out_stride: int,
                   scale: float, skip_id: int, n_rows: int, dim: int, d_grad_weight: int, grad_weight_type: int,
                   grad_weight_stride: int, accumulate: bool, stream: int) -> None:
    _check(lib().bpe_embed_grad(handle, d_ids, n_ids, d_grad_out, grad_out_type, grad_out_stride, scale, skip_id,
                                n_rows, dim, d_grad_weight, grad_weight_type, grad_weight_stride,
                                1 if accumulate else 0, stream))


def bpe_plan_blocks(handle: int, d_offsets: int | None, d_cached: int | None, n_requests: int, block_size: int,
                    d_free: int, n_free: int, d_head: int | None, d_table: int, max_blocks: int, table_stride: int,
                    d_seq_lens: int, d_slots: int, d_positions: int, n_slots: int, d_info: int, stream: int) -> None:
    _check(lib().bpe_plan_blocks(handle, d_offsets, d_cached, n_requests, block_size, d_free, n_free, d_head, d_table,
                                 max_blocks, table_stride, d_seq_lens, d_slots, d_positions, n_slots, d_info, stream))


class LogitsArgs(ctypes.Structure):
    """bpe_logits_args (device pointers as integers, None for NULL)."""
    _fields_ = [(n, t) for names, t in (
        ("logits out", ctypes.c_void_p), ("logits_type out_type", ctypes.c_int),
        ("logits_stride out_stride n_rows n_vocab", ctypes.c_int64),
        ("prompt_ids prompt_offsets", ctypes.c_void_p), ("n_prompt_ids", ctypes.c_int64),
        ("output_ids output_lens", ctypes.c_void_p), ("output_stride output_capacity", ctypes.c_int64),
        ("repetition frequency presence bias_ids bias_values bias_offsets", ctypes.c_void_p),
        ("n_bias", ctypes.c_int64), ("mask", ctypes.c_void_p), ("mask_stride n_masks", ctypes.c_int64),
        ("mask_rows", ctypes.c_void_p)) for n in names.split()]


def bpe_adjust_logits(handle: int, args: LogitsArgs, stream: int) -> None:
    _check(lib().bpe_adjust_logits(handle, ctypes.byref(args), stream))


def bpe_destroy(handle: int) -> None:
    _check(lib().bpe_destroy(handle))


# --------------------------------------------------------------- torch API --

class Tokenizer:
    """A tokenizer on one GPU. Tensors are torch CUDA tensors on that GPU;
    calls run on the current torch stream.

    All calls share one workspace on the GPU, so those made on different streams
    (an encode that prefetches beside an embed_grad, say) must not overlap: let
    one stream wait for the other, or use a Tokenizer each. Replays of a graph
    that calls were captured in count as calls; they stay valid when a later
    call outgrows the workspace, until close()."""

    def __init__(self, merges, vocab_bytes, vocab_offsets, device: int = 0):
        self.device = device
        self._lib = lib()
        self.handle = bpe_build(merges, vocab_bytes, vocab_offsets, device)

    def close(self):
        if getattr(self, "handle", None):
            bpe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @staticmethod
    def _stream():
        import torch
        return torch.cuda.current_stream().cuda_stream

    @staticmethod
    def _writes(*tensors):
        """Tells autograd that the library writes into the caller's tensors,
        which it cannot see: a graph that has saved one of them (embed saves its
        ids) refuses its backward pass from then on."""
        _torch()
        for t in tensors:
            if t.requires_grad and _torch_module.is_grad_enabled():
                raise ValueError("out: must not require a gradient")
            _increment_version(t)

    def encode_into(self, data, offsets, out_ids, out_offsets, want_total: bool = True):
        """data uint8[N], offsets int64[D + 1] -> ids written into out_ids
        (int32, capacity >= N) and out_offsets (int64[D + 1]). Returns the
        token count when want_total (that waits for the stream)."""
        self._writes(out_ids, out_offsets)
        return bpe_encode_batch(self.handle, data.data_ptr(), data.numel(), offsets.data_ptr(), offsets.numel() - 1,
                                out_ids.data_ptr(), out_ids.numel(), out_offsets.data_ptr(), want_total,
                                self._stream())

    def encode(self, data, offsets):
        """Returns (ids int32[T], out_offsets int64[D + 1]) as CUDA tensors."""
        import torch
        out_ids = torch.empty(max(1, data.numel()), dtype=torch.int32, device=data.device)
        out_off = torch.empty(offsets.numel(), dtype=torch.int64, device=data.device)
        total = self.encode_into(data, offsets, out_ids, out_off, True)
        return out_ids[:total], out_off

    def decode(self, ids, id_offsets, capacity: int | None = None):
        """Returns (bytes uint8[B], byte_offsets int64[D + 1]) as CUDA tensors."""
        import torch
        if capacity is None:
            capacity = max(1, ids.numel() * 64)
        out = torch.empty(capacity, dtype=torch.uint8, device=ids.device)
        out_off = torch.empty(id_offsets.numel(), dtype=torch.int64, device=ids.device)
        total = bpe_decode_batch(self.handle, ids.data_ptr(), ids.numel(), id_offsets.data_ptr(),
                                 id_offsets.numel() - 1, out.data_ptr(), capacity, out_off.data_ptr(), True,
                                 self._stream())
        return out[:total], out_off


    # ---- what surrounds the model ----
    # These calls take microseconds on the GPU, so their checks ask each tensor
    # for as little as they can; _refuse finds the words for what failed.

    def _refuse(self, name, t, dtypes, size=None, dims=None):
        if t.get_device() != self.device:
            raise ValueError(f"{name}: on {t.device}, the tokenizer is on cuda:{self.device}")
        if t.dtype not in dtypes:
            raise ValueError(f"{name}: {t.dtype}, need {' or '.join(str(d) for d in dtypes)}")
        if dims is not None and t.dim() != dims:
            raise ValueError(f"{name}: {t.dim()} dimensions, need {dims}")
        raise ValueError(f"{name}: needs {'adjacent elements' if size is None else f'{size} adjacent elements'}")

    def _flat(self, name, t, dtype, size):
        """The address of a tensor of `size` adjacent elements."""
        if t.dtype is not dtype or t.get_device() != self.device or t.numel() != size or not t.is_contiguous():
            self._refuse(name, t, (dtype,), size)
        return t.data_ptr()

    def plan_blocks(self, offsets, cached, table, free, block_size: int, n_slots: int | None = None, head=None):
        """Block tables, cache slots and positions for the next step of a
        batch of requests (see bpe_plan_blocks): offsets int64[n + 1] of the
        packed new tokens, or None for one new token each; cached int32[n]
        tokens in the cache, or None; table int32[n, max_blocks], extended in
        place from the free list int32[m], of which the first head (int64[1],
        None: 0) entries are taken. n_slots: places for the new tokens, at
        least their number (needed with offsets, whose end is on the device).
        Returns (seq_lens int32[n], slots int64[n_slots], positions
        int32[n_slots], info int64[2]: head after the call, blocks lacking)."""
        torch, flat = _torch(), self._flat
        i32, i64 = _int32, _int64
        if table.dtype is not i32 or table.get_device() != self.device or table.dim() != 2:
            self._refuse("table", table, (i32,), dims=2)
        n, width = table.shape
        stride, step = table.stride()
        if step != 1 and width > 1:
            raise ValueError("table: the elements of a row must be adjacent")
        if n_slots is None:
            if offsets is not None:
                raise ValueError("n_slots: the number of new tokens (or more) is needed with offsets")
            n_slots = n
        n_free = free.numel()
        p_offsets = None if offsets is None else flat("offsets", offsets, i64, n + 1)
        p_cached = None if cached is None else flat("cached", cached, i32, n)
        p_free = flat("free", free, i32, n_free)
        p_head = None if head is None else flat("head", head, i64, 1)
        self._writes(table)
        empty, dev = torch.empty, table.device
        seq_lens = empty(n, dtype=i32, device=dev)
        slots = empty(n_slots, dtype=i64, device=dev)
        positions = empty(n_slots, dtype=i32, device=dev)
        info = empty(2, dtype=i64, device=dev)
        rc = self._lib.bpe_plan_blocks(self.handle, p_offsets, p_cached, n, block_size, p_free, n_free, p_head,
                                       table.data_ptr(), width, stride, seq_lens.data_ptr(), slots.data_ptr(),
                                       positions.data_ptr(), n_slots, info.data_ptr(), _raw_stream(self.device))
        if rc:
            _check(rc)
        return seq_lens, slots, positions, info

    def adjust_logits(self, logits, prompt=None, output=None, repetition=None, frequency=None, presence=None,
                      bias=None, mask=None, mask_rows=None, dtype=None, out=None):
        """Penalties for repeated tokens, biases and grammar masks (see
        bpe_adjust_logits) on logits [n, vocab] in 32 or 16 bits, into a new
        tensor of logits' type or ``dtype``, or into ``out`` (which may be
        logits). prompt: (ids int32[p], offsets int64[n + 1]) as encode
        returns them; output: (ids int32[n, capacity], lens int32[n]);
        repetition, frequency, presence: float32[n]; bias: (ids int32[m],
        values float32[m], offsets int64[n + 1]); mask: int32 or uint32
        [masks, ceil(vocab / 32)], bit v % 32 of word v / 32 set for an
        allowed token; mask_rows: int32[n], each row's mask or -1, needs mask
        (which may have no rows where all are -1). An empty list of prompt,
        output or bias ids counts as left out. Has no derivative: a backward pass through its result raises, and ``out`` is
        refused for inputs that torch records derivatives of."""
        torch, types, flat = _torch(), _type_codes, self._flat
        i32, i64, f32 = _int32, _int64, _float32
        if _tracked(logits, repetition, frequency, presence, None if bias is None else bias[1]):
            if out is not None:
                raise ValueError("out: adjust_logits has no derivative, so it needs inputs without one "
                                 "(torch.no_grad or detach)")
            return _functions()[2].apply(
                lambda: self.adjust_logits(logits, prompt, output, repetition, frequency, presence, bias, mask,
                                           mask_rows, dtype), logits, repetition, frequency, presence,
                None if bias is None else bias[1])
        code = types.get(logits.dtype)
        if code is None or logits.get_device() != self.device or logits.dim() != 2:
            self._refuse("logits", logits, types, dims=2)
        n, vocab = logits.shape
        stride, step = logits.stride()
        if step != 1 and vocab > 1:
            if out is logits:
                raise ValueError("out: the elements of a row must be adjacent")
            logits = logits.contiguous()
            stride = vocab
        if out is None:
            out = torch.empty((n, vocab), dtype=dtype or logits.dtype, device=logits.device)
            out_stride = vocab
        else:
            if out.get_device() != self.device or out.dim() != 2:
                self._refuse("out", out, types, dims=2)
            out_stride, step = out.stride()
            if out.shape != logits.shape or (step != 1 and vocab > 1):
                raise ValueError("out: needs the shape of logits, the elements of a row adjacent")
            self._writes(out)
            if dtype is not None and dtype is not out.dtype:
                raise ValueError(f"out: {out.dtype}, but dtype is {dtype}")
        out_code = types.get(out.dtype)
        if out_code is None:
            self._refuse("out", out, types)
        p_ids = p_off = o_ids = o_lens = b_ids = b_values = b_off = p_mask = p_rows = 0
        n_prompt = o_stride = o_cap = n_bias = m_stride = n_masks = 0
        if prompt is not None:
            ids, offsets = prompt
            n_prompt = ids.numel()
            p_ids, p_off = flat("prompt ids", ids, i32, n_prompt), flat("prompt offsets", offsets, i64, n + 1)
        if output is not None:
            ids, lens = output
            if ids.dtype is not i32 or ids.get_device() != self.device or ids.dim() != 2:
                self._refuse("output ids", ids, (i32,), dims=2)
            o_stride, step = ids.stride()
            rows, o_cap = ids.shape
            if rows != n or (step != 1 and o_cap > 1):
                raise ValueError("output ids: needs a row for each row of logits, its elements adjacent")
            o_ids, o_lens = ids.data_ptr(), flat("output lens", lens, i32, n)
        p_rep = 0 if repetition is None else flat("repetition", repetition, f32, n)
        p_freq = 0 if frequency is None else flat("frequency", frequency, f32, n)
        p_pres = 0 if presence is None else flat("presence", presence, f32, n)
        if bias is not None:
            ids, values, offsets = bias
            n_bias = ids.numel()
            b_ids, b_values = flat("bias ids", ids, i32, n_bias), flat("bias values", values, f32, n_bias)
            b_off = flat("bias offsets", offsets, i64, n + 1)
        if mask is not None:
            if (mask.dtype is not i32 and mask.dtype is not torch.uint32) or mask.get_device() != self.device \
                    or mask.dim() != 2:
                self._refuse("mask", mask, (i32, torch.uint32), dims=2)
            n_masks, words = mask.shape
            m_stride, step = mask.stride()
            if words < (vocab + 31) // 32 or (step != 1 and words > 1):
                raise ValueError("mask: needs a bit for each token, the words of a row adjacent")
            p_mask = mask.data_ptr()
            if mask_rows is not None:
                p_rows = flat("mask rows", mask_rows, i32, n)
            if not n_masks and n:
                # torch gives an empty tensor no address, and without one the call would take every token as allowed
                if mask_rows is None:
                    raise BpeError(1, "adjust_logits: fewer masks than rows, and no mask_rows")
                p_mask = p_rows
        elif mask_rows is not None:
            raise ValueError("mask_rows: there is no mask")
        rc = self._lib.bpe_adjust_logits(
            self.handle,
            _pack_logits(logits.data_ptr(), out.data_ptr(), code, out_code, stride, out_stride, n, vocab, p_ids, p_off,
                         n_prompt, o_ids, o_lens, o_stride, o_cap, p_rep, p_freq, p_pres, b_ids, b_values, b_off,
                         n_bias, p_mask, m_stride, n_masks, p_rows), _raw_stream(self.device))
        if rc:
            _check(rc)
        return out

    def embed(self, ids, weight, scale: float = 1.0, skip_id: int | None = None, dtype=None, out=None):
        """scale * weight[ids] in weight's type, or in ``dtype``: ids int32 of
        any shape, weight [rows, dim] in 32 or 16 bits with any row stride.
        Tokens equal to skip_id get zeros. Differentiable with respect to
        weight in backward and forward mode, as often as wanted (its gradient
        runs embed_grad), unless ``out`` is given."""
        torch, types, device = _torch(), _type_codes, self.device
        code = types.get(weight.dtype)
        if code is None or weight.get_device() != device or weight.dim() != 2:
            self._refuse("weight", weight, types, dims=2)
        if ids.dtype is not _int32 or ids.get_device() != device:
            self._refuse("ids", ids, (_int32,))
        if not ids.is_contiguous():
            ids = ids.contiguous()
        n_rows, dim = weight.shape
        stride, step = weight.stride()
        shape = (*ids.shape, dim)
        out_stride = dim
        if out is None:
            if _tracked(weight):
                return _functions()[0].apply(self, ids, weight, scale, skip_id, dtype or weight.dtype)
            out = torch.empty(shape, dtype=dtype or weight.dtype, device=weight.device)
        else:
            if out.get_device() != device or out.shape != shape:
                raise ValueError("out: needs the shape of ids and weight's columns, on the tokenizer's device")
            if len(shape) == 2:
                out_stride, out_step = out.stride()
                if out_step != 1 and dim > 1:
                    raise ValueError("out: the elements of a row must be adjacent")
            elif not out.is_contiguous():
                raise ValueError("out: needs to be contiguous where ids is not one-dimensional")
            self._writes(out)
            if dtype is not None and dtype is not out.dtype:
                raise ValueError(f"out: {out.dtype}, but dtype is {dtype}")
        out_code = types.get(out.dtype)
        if out_code is None:
            self._refuse("out", out, types)
        if step != 1 and dim > 1:
            weight = weight.contiguous()
            stride = dim
        rc = self._lib.bpe_embed(self.handle, ids.data_ptr(), ids.numel(), weight.data_ptr(), code, n_rows, dim, stride,
                                 scale, _skip(skip_id), out.data_ptr(), out_code, out_stride, _raw_stream(device))
        if rc:
            _check(rc)
        return out

    def embed_grad(self, ids, grad, n_rows: int, scale: float = 1.0, skip_id: int | None = None, dtype=None,
                   out=None, accumulate: bool = False):
        """The gradient [n_rows, dim] of embed's weight for the gradient
        ``grad`` [*ids.shape, dim] of its result, in grad's type or in
        ``dtype``, or written into (accumulate: added to) ``out``.
        Differentiable with respect to grad unless ``out`` is given."""
        torch, types, device = _torch(), _type_codes, self.device
        code = types.get(grad.dtype)
        if code is None or grad.get_device() != device:
            self._refuse("grad", grad, types)
        if ids.dtype is not _int32 or ids.get_device() != device:
            self._refuse("ids", ids, (_int32,))
        if not ids.is_contiguous():
            ids = ids.contiguous()
        n = ids.numel()
        shape = grad.shape
        dim = shape[-1]
        if shape[:-1] != ids.shape:
            raise ValueError("grad: needs the shape of ids and one more dimension")
        if out is None and not accumulate and _tracked(grad):
            return _functions()[1].apply(self, ids, grad, n_rows, scale, skip_id, dtype or grad.dtype)
        if len(shape) != 2:
            grad = grad.reshape(n, dim)
        stride, step = grad.stride()
        if step != 1 and dim > 1:
            grad = grad.contiguous()
            stride = dim
        if out is None:
            if accumulate:
                raise ValueError("accumulate needs out")
            out = torch.empty((n_rows, dim), dtype=dtype or grad.dtype, device=grad.device)
            out_stride = dim
        else:
            if out.get_device() != device or out.dim() != 2:
                self._refuse("out", out, types, dims=2)
            out_stride, step = out.stride()
            if out.shape != (n_rows, dim) or (step != 1 and dim > 1):
                raise ValueError("out: needs n_rows rows of grad's columns, the elements of a row adjacent")
            self._writes(out)
            if dtype is not None and dtype is not out.dtype:
                raise ValueError(f"out: {out.dtype}, but dtype is {dtype}")
        out_code = types.get(out.dtype)
        if out_code is None:
            self._refuse("out", out, types)
        rc = self._lib.bpe_embed_grad(self.handle, ids.data_ptr(), n, grad.data_ptr(), code, stride, scale,
                                      _skip(skip_id), n_rows, dim, out.data_ptr(), out_code,
                                      out_stride, accumulate, _raw_stream(device))
        if rc:
            _check(rc)
        return out


def _skip(skip_id):
    """skip_id for the library, in 32 bits: ctypes would cut what is longer, and skip another id."""
    if skip_id is None:
        return NO_ID
    if not -2 ** 31 <= skip_id < 2 ** 31:
        raise ValueError(f"skip_id: {skip_id} is no int32")
    return skip_id


# bpe_logits_args in native layout, for Tokenizer.adjust_logits: one pack takes
# a tenth of the time of filling a LogitsArgs field by field
_pack_logits = struct.Struct("@PPiiqqqqPPqPPqqPPPPPPqPqqP").pack

_type_codes = {}  # torch dtype -> BPE_* code

_torch_module = _int32 = _int64 = _float32 = _raw_stream = _forward_ad = _increment_version = None


def _torch():
    """torch, imported on first use, with what the calls above take from it."""
    global _torch_module, _int32, _int64, _float32, _raw_stream, _forward_ad, _increment_version
    if _torch_module is None:
        import torch
        _int32, _int64, _float32 = torch.int32, torch.int64, torch.float32
        _raw_stream = torch._C._cuda_getCurrentRawStream
        _forward_ad = torch.autograd.forward_ad
        _increment_version = torch.autograd.graph.increment_version
        _type_codes.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16})
        _torch_module = torch
    return _torch_module


def _tracked(*tensors):
    """Whether torch records derivatives, backward or forward, of one of the
    tensors (or Nones)."""
    if _torch_module.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    if _forward_ad._current_level >= 0:
        for t in tensors:
            if t is not None and _forward_ad.unpack_dual(t).tangent is not None:
                return True
    return False


def _functions():
    """The autograd functions of Tokenizer.embed, embed_grad and adjust_logits
    (made once: torch is imported on first use only). The first two are linear
    and each other's adjoint, so their derivatives of any order, backward and
    forward, are calls of the two. The last has none, and says so when one is
    asked for."""
    global _function_list
    if _function_list is None:
        import torch

        class Embed(torch.autograd.Function):
            @staticmethod
            def forward(ctx, tok, ids, weight, scale, skip_id, dtype):
                ctx.args = (tok, weight.shape[0], scale, skip_id, weight.dtype, dtype)
                ctx.save_for_backward(ids)
                ctx.save_for_forward(ids)
                return tok.embed(ids, weight.detach(), scale, skip_id, dtype)

            @staticmethod
            def backward(ctx, grad):
                tok, n_rows, scale, skip_id, dtype, _ = ctx.args
                (ids,) = ctx.saved_tensors
                return None, None, tok.embed_grad(ids, grad, n_rows, scale, skip_id, dtype), None, None, None

            @staticmethod
            def jvp(ctx, _tok, _ids, weight, *_):
                tok, _, scale, skip_id, _, dtype = ctx.args
                (ids,) = ctx.saved_tensors
                return tok.embed(ids, weight, scale, skip_id, dtype)

        class EmbedGrad(torch.autograd.Function):
            @staticmethod
            def forward(ctx, tok, ids, grad, n_rows, scale, skip_id, dtype):
                ctx.args = (tok, n_rows, scale, skip_id, grad.dtype, dtype)
                ctx.save_for_backward(ids)
                ctx.save_for_forward(ids)
                return tok.embed_grad(ids, grad.detach(), n_rows, scale, skip_id, dtype)

            @staticmethod
            def backward(ctx, grad):
                tok, _, scale, skip_id, dtype, _ = ctx.args
                (ids,) = ctx.saved_tensors
                return None, None, tok.embed(ids, grad, scale, skip_id, dtype), None, None, None, None

            @staticmethod
            def jvp(ctx, _tok, _ids, grad, *_):
                tok, n_rows, scale, skip_id, _, dtype = ctx.args
                (ids,) = ctx.saved_tensors
                return tok.embed_grad(ids, grad, n_rows, scale, skip_id, dtype)

        class AdjustLogits(torch.autograd.Function):
            @staticmethod
            def forward(ctx, call, *inputs):
                return call()

            @staticmethod
            def backward(ctx, grad):
                raise RuntimeError("adjust_logits has no gradient")

            @staticmethod
            def jvp(ctx, *tangents):
                raise RuntimeError("adjust_logits has no derivative")

        _function_list = Embed, EmbedGrad, AdjustLogits
    return _function_list


_function_list = None


def pretokenize(data, offsets):
    """Start bits (uint32[(N + 31) / 32]) of the pre-tokens of a batch."""
    import torch
    words = max(1, (data.numel() + 31) // 32)
    bits = torch.zeros(words, dtype=torch.int32, device=data.device)
    bpe_pretokenize_batch(data.data_ptr(), data.numel(), offsets.data_ptr(), offsets.numel() - 1, bits.data_ptr(),
                          torch.cuda.current_stream().cuda_stream)
    return bits
