"""Penalties, biases and masks on logits against a 64-bit computation.

Bound: with m biases for a token the 32-bit computation makes one division or
product, one product, two subtractions and m additions, each off by at most
2^-24 of the sum of magnitudes involved: (m + 5) 2^-24 (|x rho| or |x / rho| +
|frequency| k + |presence| + sum|bias|), and the result is rounded once.
"""
import numpy as np
import pytest

from tests.ops_util import assert_close, byte_tokenizer, load

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def bpe():
    return load()


@pytest.fixture(scope="module")
def tok(bpe):
    t = byte_tokenizer(bpe)
    yield t
    t.close()


def dtypes():
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def make(n, vocab, prompt, output, bias, masks, seed, dtype="f32", hot=None):
    """Inputs on the GPU. hot: ids are drawn from the first `hot` tokens, so that they repeat."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    top = min(vocab, hot or vocab)

    def ids(*shape):
        x = torch.randint(0, top, shape, generator=g, device="cuda", dtype=torch.int32)
        return x if hot is None else (x * 37 % vocab).to(torch.int32)

    def cuts(total):
        c = torch.randint(0, total + 1, (n - 1,), generator=g, device="cuda").sort().values
        return torch.cat([c.new_zeros(1), c, c.new_full((1,), total)])

    s = {"logits": (torch.randn(n, vocab, generator=g, device="cuda") * 4).to(dtypes()[dtype])}
    if prompt is not None:
        s["prompt"] = (ids(n * prompt), cuts(n * prompt))
    if output is not None:
        s["output"] = (ids(n, output + 3), torch.randint(0, output + 1, (n,), generator=g, device="cuda",
                                                         dtype=torch.int32))
    s["repetition"] = torch.rand(n, generator=g, device="cuda") + 0.6
    s["frequency"] = torch.rand(n, generator=g, device="cuda") - 0.3
    s["presence"] = torch.rand(n, generator=g, device="cuda") - 0.3
    if bias is not None:
        s["bias"] = (ids(n * bias), torch.randn(n * bias, generator=g, device="cuda") * 3, cuts(n * bias))
    if masks:
        s["mask"] = torch.randint(-2 ** 31, 2 ** 31, (masks, (vocab + 31) // 32), generator=g, device="cuda").to(
            torch.int32)
        s["mask_rows"] = torch.randint(-1, masks, (n,), generator=g, device="cuda", dtype=torch.int32)
    return s


def plain(s):
    """(values, bounds) in 64 bits."""
    import torch
    h = {k: (tuple(t.cpu().numpy() for t in v) if isinstance(v, tuple) else v.cpu()) for k, v in s.items()
         if v is not None}
    x = h["logits"].double().numpy().copy()
    n, vocab = x.shape
    mag, terms = np.zeros_like(x), np.zeros_like(x)
    inside = lambda ids: ids[(ids >= 0) & (ids < vocab)]  # noqa: E731
    with np.errstate(all="ignore"):
        for b in range(n):
            k = np.zeros(vocab)
            if "output" in h:
                np.add.at(k, inside(h["output"][0][b, :h["output"][1][b]]), 1)
            seen = k > 0
            if "prompt" in h:
                lo, hi = h["prompt"][1][b:b + 2]
                seen[inside(h["prompt"][0][lo:hi])] = True
            rho = float(h["repetition"][b]) if "repetition" in h else 1.0
            phi = float(h["frequency"][b]) if "frequency" in h else 0.0
            pi = float(h["presence"][b]) if "presence" in h else 0.0
            x[b, seen] = np.where(x[b, seen] > 0, x[b, seen] / rho, x[b, seen] * rho)
            said = k > 0
            x[b, said] -= phi * k[said] + pi
            mag[b] = np.abs(x[b]) + 2 * (abs(phi) * k + abs(pi) * said)
            if "bias" in h:
                lo, hi = h["bias"][2][b:b + 2]
                ids, values = h["bias"][0][lo:hi], h["bias"][1][lo:hi].astype(np.float64)
                ok = (ids >= 0) & (ids < vocab)
                np.add.at(x[b], ids[ok], values[ok])
                np.add.at(mag[b], ids[ok], np.abs(values[ok]))
                np.add.at(terms[b], ids[ok], 1)
            mag[b][~seen & (terms[b] == 0)] = 0
            if "mask" in h:
                row = int(h["mask_rows"][b]) if "mask_rows" in h else b
                if row >= 0:
                    bits = np.unpackbits(h["mask"][row].numpy().view(np.uint8), bitorder="little")[:vocab]
                    x[b, bits == 0] = -np.inf
    return torch.from_numpy(x), torch.from_numpy(np.nan_to_num((terms + 5) * EPS * mag, nan=0.0, posinf=0.0))


def call(tok, s, **more):
    return tok.adjust_logits(s["logits"], **{k: v for k, v in s.items() if k != "logits"}, **more)


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32"),
                                       ("f16", "f32"), ("f32", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("n,vocab,prompt,output,bias,masks", [
    (1, 1, 1, 1, 1, 1), (1, 31, 3, 0, 0, 0), (3, 33, 5, 4, 2, 2), (2, 768, 50, 20, 5, 1), (5, 4096, 0, 40, 0, 0),
    (4, 4097, 100, 0, 0, 3), (7, 10_001, 300, 100, 30, 7), (2, 70_003, 2000, 500, 100, 1), (40, 1000, 7, 3, 1, 11)])
def test_all_parts(tok, dtype, out, n, vocab, prompt, output, bias, masks):
    s = make(n, vocab, prompt, output, bias, masks, vocab + n, dtype)
    want, bound = plain(s)
    assert_close(call(tok, s, dtype=dtypes()[out]), want, bound, "all parts")


@pytest.mark.parametrize("parts", ["", "prompt", "output", "bias", "mask", "prompt output", "bias mask",
                                   "output mask", "prompt bias"])
@pytest.mark.parametrize("vocab", [63, 9000])
def test_parts_left_out(tok, parts, vocab):
    import torch
    has = parts.split()
    s = make(6, vocab, 40 if "prompt" in has else None, 30 if "output" in has else None,
             10 if "bias" in has else None, 4 if "mask" in has else 0, 5)
    want, bound = plain(s)
    got = call(tok, s)
    assert_close(got, want, bound, parts)
    if not has:
        assert torch.equal(got, s["logits"])
    for left in ("repetition", "frequency", "presence"):
        t = dict(s)
        t[left] = None
        want, bound = plain(t)
        assert_close(call(tok, t), want, bound, f"{parts} without {left}")
    t = dict(s)
    t["repetition"], t["frequency"], t["presence"] = (torch.full_like(s["presence"], v) for v in (1.0, 0.0, 0.0))
    want, bound = plain(t)
    assert_close(call(tok, t), want, bound, f"{parts} neutral")


@pytest.mark.parametrize("prompt,output,bias,hot", [(3000, 3000, 300, 5), (0, 70_001, 0, 1), (70_001, 9, 0, 900),
                                                    (20_000, 20_000, 1000, 1000)])
def test_long_and_repeated_history(tok, prompt, output, bias, hot):
    s = make(3, 32_256, prompt, output, bias, 0, hot, hot=hot)
    want, bound = plain(s)
    assert_close(call(tok, s), want, bound, "repeated")
    assert (call(tok, s) == call(tok, s)).all()


@pytest.mark.parametrize("n,vocab,prompt,output,bias,masks,hot", [
    (400, 9001, 60, 30, 5, 400, None), (80, 32_256, 9000, 50, 0, 0, None), (90, 32_256, 200, 12_000, 300, 3, None),
    (350, 8200, 3000, 100, 0, 2, 40), (310, 5000, 0, 0, 700, 0, 300), (320, 8000, 40, 0, 0, 1, None)])
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f32", "f32"), ("f16", "f16")])
def test_many_rows(tok, n, vocab, prompt, output, bias, masks, hot, dtype, out):
    s = make(n, vocab, prompt, output, bias, masks, n + vocab, dtype, hot=hot)
    want, bound = plain(s)
    assert_close(call(tok, s, dtype=dtypes()[out]), want, bound, "many rows")
    if dtype == out:
        assert_close(call(tok, s, out=s["logits"]), want, bound, "many rows in place")


def test_one_row_takes_all_of_the_history(tok):
    import torch
    s = make(6, 5000, 100, 20, 20, 0, 9)
    for name in ("prompt", "bias"):
        *ids, off = s[name]
        off = torch.where(torch.arange(7, device="cuda") < 4, 0, ids[0].numel())
        s[name] = (*ids, off)
    want, bound = plain(s)
    assert_close(call(tok, s), want, bound, "one row")


def test_masks(tok):
    import torch
    s = make(5, 1003, 20, 20, 5, 5, 11)
    s["mask"][0] = 0    # nothing is allowed
    s["mask"][1] = -1   # everything is
    s["mask"][2] = 0
    s["mask"][2, 31] = 1 << 10  # the last token alone
    del s["mask_rows"]
    s["logits"][3, ::7] = float("nan")
    s["logits"][3, 1::7] = float("inf")
    s["logits"][3, 2::7] = torch.finfo(torch.float32).min
    s["logits"][4, ::5] = float("-inf")
    want, bound = plain(s)
    got = call(tok, s)
    assert_close(got, want, bound, "masks")
    assert bool((got[0] == float("-inf")).all())
    assert int((got[2] > float("-inf")).sum()) == 1 and bool(got[2, 1002] > float("-inf"))
    # more masks than rows, one mask for all, words past the vocabulary, unsigned words
    s["mask"] = torch.cat([s["mask"], torch.full_like(s["mask"][:, :3], -1)], 1)
    assert torch.equal(call(tok, s).nan_to_num(3.0), got.nan_to_num(3.0))
    s["mask_rows"] = torch.zeros(5, dtype=torch.int32, device="cuda")
    s["mask"] = s["mask"][2:3].view(torch.uint32)
    got = call(tok, s)
    assert int((got > float("-inf")).sum()) <= 5


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_infinities_and_lowest_values(tok, dtype):
    import torch
    s = make(4, 600, 200, 100, 30, 0, 12, dtype)
    x = s["logits"]
    x[0, ::3], x[1, ::4], x[2, ::5] = float("-inf"), float("inf"), float("nan")
    s["repetition"][3] = 1.0
    s["frequency"][3], s["presence"][3] = 0.0, 0.0
    x[3] = torch.finfo(x.dtype).min
    s["bias"] = (s["bias"][0], s["bias"][1].abs(), s["bias"][2])  # the lowest value and more: no overflow
    want, bound = plain(s)
    assert_close(call(tok, s, dtype=torch.float32), want, bound, "special")
    s["bias"][1].fill_(float("-inf"))
    want, bound = plain(s)
    assert_close(call(tok, s, dtype=torch.float32), want, bound, "banned")


def test_token_zero_and_untouched_bits(tok):
    """Tokens that nothing concerns keep their bits."""
    import torch
    s = make(3, 4099, 5, 5, 2, 0, 13, "bf16")
    got = call(tok, s)
    want, bound = plain(s)
    assert_close(got, want, bound, "bits")
    free = torch.ones_like(got, dtype=torch.bool)
    for b in range(3):
        for ids in (s["prompt"][0][s["prompt"][1][b]:s["prompt"][1][b + 1]], s["output"][0][b, :s["output"][1][b]],
                    s["bias"][0][s["bias"][2][b]:s["bias"][2][b + 1]]):
            free[b, ids.long()] = False
    assert torch.equal(got[free], s["logits"][free])


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("vocab,first,stride,out_first,out_stride", [
    (1000, 1, 1003, 0, 1000), (1000, 0, 1008, 3, 1001), (5001, 2, 5003, 2, 5003), (4096, 5, 4096, 5, 4096),
    (37, 0, 0, 0, 40)])
def test_strides(tok, dtype, out, vocab, first, stride, out_first, out_stride):
    import torch
    n = 4
    s = make(n, vocab, 50, 30, 5, 3, 14, dtype)
    base = torch.randn(first + n * max(stride, 1) + vocab, device="cuda").to(dtypes()[dtype])
    s["logits"] = torch.as_strided(base, (n, vocab), (stride, 1), first)
    whole = torch.full((out_first + n * out_stride + 9,), 77.0, device="cuda", dtype=dtypes()[out])
    view = torch.as_strided(whole, (n, vocab), (out_stride, 1), out_first)
    want, bound = plain(s)
    assert_close(call(tok, s, out=view), want, bound, "strides")
    rest = torch.ones_like(whole, dtype=torch.bool)
    torch.as_strided(rest, (n, vocab), (out_stride, 1), out_first).fill_(False)
    assert bool((whole[rest] == 77.0).all())
    cols = s["logits"].t().contiguous().t()  # columns apart
    assert_close(tok.adjust_logits(cols, **{k: v for k, v in s.items() if k != "logits"}), want, bound, "columns")
    wide = torch.zeros(n, 64, dtype=torch.int32, device="cuda")
    wide[:, 7:7 + s["output"][0].shape[1]] = s["output"][0]
    s["output"] = (wide[:, 7:7 + s["output"][0].shape[1]], s["output"][1])
    assert_close(call(tok, s, out=view), want, bound, "output rows apart")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place(tok, dtype):
    import torch
    s = make(5, 9001, 100, 50, 20, 3, 15, dtype)
    want = call(tok, s)
    got = call(tok, s, out=s["logits"])
    assert got is s["logits"] and torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("first,stride", [(0, 40_000), (1, 40_003), (3, 40_001)])
def test_in_place_without_masks(tok, dtype, first, stride):
    """Only the tokens that the history or a bias concerns are touched."""
    import torch
    n, vocab = 5, 40_000
    s = make(n, vocab, 900, 300, 40, 0, 25, dtype)
    whole = torch.randn(first + n * stride, device="cuda").to(dtypes()[dtype])
    before = whole.clone()
    view = torch.as_strided(whole, (n, vocab), (stride, 1), first)
    s["logits"] = view.clone()
    want = call(tok, s)
    s["logits"] = view
    assert call(tok, s, out=view) is view
    assert torch.equal(view, want)
    torch.as_strided(before, (n, vocab), (stride, 1), first).copy_(want)
    assert torch.equal(whole, before)
    nothing = {"logits": view, "mask": None}
    assert torch.equal(call(tok, nothing, out=view), want)


def test_logits_past_2_to_the_31_elements(tok):
    import torch
    n, vocab = 20_000, 113_645  # 2.27e9 elements
    x = torch.zeros(n, vocab, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(vocab, device="cuda").to(torch.bfloat16)
    x[-1] = last
    off = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
    off[-1] = 2
    ids = torch.tensor([vocab - 1, 5], dtype=torch.int32, device="cuda")
    vals = torch.tensor([2.0, -3.0], device="cuda")
    tok.adjust_logits(x, bias=(ids, vals, off), out=x)
    last = last.float()
    last[ids.long()] += vals
    assert torch.equal(x[-1], last.to(torch.bfloat16)) and not bool(x[n - 2].any()) and not bool(x[0].any())


def _status(bpe, tok):
    import torch
    try:
        bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)
    except bpe.BpeError as e:
        return e.code
    return 0


def test_what_is_out_of_range_is_left_out(bpe, tok):
    import torch
    s = make(4, 900, 30, 20, 10, 2, 16)
    want, bound = plain(s)
    assert_close(call(tok, s), want, bound, "in range")
    assert _status(bpe, tok) == 0
    for name in ("prompt", "output", "bias"):
        for bad in (900, -1, 2 ** 31 - 1):
            t = dict(s)
            ids = s[name][0].clone()
            ids.reshape(-1)[::5] = bad
            t[name] = (ids, *s[name][1:])
            if name == "output":
                t["output"] = (ids, torch.full_like(s["output"][1], 20))
            want, bound = plain(t)
            assert_close(call(tok, t), want, bound, name)
            assert _status(bpe, tok) == 7 and _status(bpe, tok) == 0
    # lengths and offsets that leave their lists: the row's part is left out
    t = dict(s)
    lens = s["output"][1].clone()
    lens[1], lens[2] = 24, -1
    t["output"] = (s["output"][0], lens)
    u = dict(s)
    u["output"] = (s["output"][0], torch.where((lens > 23) | (lens < 0), 0, lens))
    want, bound = plain(u)
    assert_close(call(tok, t), want, bound, "lens")
    assert _status(bpe, tok) == 7
    for name in ("prompt", "bias"):
        t, u = dict(s), dict(s)
        ids, off = s[name][0], s[name][-1].clone()
        off[4] = ids.numel() + 1  # row 3
        t[name] = (*s[name][:-1], off)
        fixed = s[name][-1].clone()
        fixed[4] = fixed[3]
        u[name] = (*s[name][:-1], fixed)
        want, bound = plain(u)
        assert_close(call(tok, t), want, bound, name)
        assert _status(bpe, tok) == 7
    t, u = dict(s), dict(s)
    rows = s["mask_rows"].clone()
    rows[0], rows[1] = 2, -2
    t["mask_rows"], u["mask_rows"] = rows, torch.where((rows > 1) | (rows < -1), -1, rows)
    want, bound = plain(u)
    assert_close(call(tok, t), want, bound, "mask rows")
    assert _status(bpe, tok) == 7 and _status(bpe, tok) == 0


def test_nothing(tok):
    import torch
    assert tok.adjust_logits(torch.zeros(0, 50, device="cuda")).shape == (0, 50)
    assert tok.adjust_logits(torch.zeros(3, 0, device="cuda")).shape == (3, 0)


def test_other_streams_and_capture(tok):
    import torch
    s = make(9, 20_000, 300, 100, 30, 4, 17, "bf16")
    want = call(tok, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(tok, s)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(tok, s, out=out)
    s["logits"].neg_()
    s["output"][1].fill_(7)
    graph.replay()
    want, bound = plain(s)
    assert_close(out, want, bound, "replayed")


def test_refusals(bpe, tok):
    import ctypes
    import torch
    s = make(3, 100, 10, 10, 4, 3, 18)
    L, st = bpe.lib(), torch.cuda.current_stream().cuda_stream

    def args(**change):
        a = bpe.LogitsArgs(
            logits=s["logits"].data_ptr(), out=s["logits"].data_ptr(), logits_stride=100, out_stride=100, n_rows=3,
            n_vocab=100, prompt_ids=s["prompt"][0].data_ptr(), prompt_offsets=s["prompt"][1].data_ptr(),
            n_prompt_ids=30, output_ids=s["output"][0].data_ptr(), output_lens=s["output"][1].data_ptr(),
            output_stride=13, output_capacity=13, repetition=s["repetition"].data_ptr(),
            frequency=s["frequency"].data_ptr(), presence=s["presence"].data_ptr(), bias_ids=s["bias"][0].data_ptr(),
            bias_values=s["bias"][1].data_ptr(), bias_offsets=s["bias"][2].data_ptr(), n_bias=12,
            mask=s["mask"].data_ptr(), mask_stride=4, n_masks=3, mask_rows=s["mask_rows"].data_ptr())
        for k, v in change.items():
            setattr(a, k, v)
        return ctypes.byref(a)

    assert L.bpe_adjust_logits(tok.handle, args(), st) == 0
    assert L.bpe_adjust_logits(None, args(), st) == 1
    assert L.bpe_adjust_logits(tok.handle, None, st) == 1
    for change in ({"logits": None}, {"out": None}, {"logits_type": 3}, {"out_type": -1}, {"logits_stride": -100},
                   {"out_stride": 99}, {"n_rows": -1}, {"n_rows": 65536}, {"n_vocab": -1}, {"n_vocab": 2 ** 31},
                   {"prompt_offsets": None}, {"n_prompt_ids": -1}, {"output_lens": None}, {"output_stride": -1},
                   {"output_capacity": -1}, {"output_capacity": 2 ** 30}, {"bias_values": None},
                   {"bias_offsets": None}, {"n_bias": -1}, {"mask_stride": 3}, {"n_masks": -1},
                   {"mask_rows": None, "n_masks": 2}, {"out_type": 1}, {"logits_stride": 101},
                   {"logits": s["logits"].data_ptr() + 2}, {"out": s["logits"].data_ptr() + 1},
                   {"prompt_ids": s["prompt"][0].data_ptr() + 2}, {"prompt_offsets": s["prompt"][1].data_ptr() + 4},
                   {"output_lens": s["output"][1].data_ptr() + 1}, {"bias_values": s["bias"][1].data_ptr() + 2},
                   {"mask": s["mask"].data_ptr() + 2}, {"mask_rows": s["mask_rows"].data_ptr() + 1},
                   {"repetition": s["repetition"].data_ptr() + 3}):
        assert L.bpe_adjust_logits(tok.handle, args(**change), st) == 1, change
        assert b"bpe_adjust_logits" in L.bpe_last_error()
    x = s["logits"]
    for more in ({"prompt": (s["prompt"][0].long(), s["prompt"][1])}, {"prompt": (s["prompt"][0], s["prompt"][1][1:])},
                 {"output": (s["output"][0][:2], s["output"][1])}, {"output": (s["output"][0], s["output"][1].long())},
                 {"repetition": s["repetition"].double()}, {"presence": s["presence"][:2]},
                 {"bias": (s["bias"][0], s["bias"][1][1:], s["bias"][2])}, {"mask": s["mask"][:, :3]},
                 {"mask": s["mask"].long()}, {"mask": s["mask"], "mask_rows": s["mask_rows"].cpu()},
                 {"out": torch.zeros(3, 101, device="cuda")}, {"dtype": torch.float64}):
        with pytest.raises(ValueError):
            tok.adjust_logits(x, **more)
    with pytest.raises(ValueError):
        tok.adjust_logits(x[0])
    with pytest.raises(ValueError):
        tok.adjust_logits(x.cpu())
