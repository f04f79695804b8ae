"""Keys and values into a cache in 4 bits and back, byte for byte against the
layout and the rounding that the header states."""
import numpy as np
import pytest

from tests import paged_util as pu
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


def status(bpe, tok):
    import torch
    bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)


def rows(shape, dtype, seed=0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-6, 7, shape[:-1], generator=g, device="cuda").float())[..., None]
    return (x + torch.randn(shape[-1], generator=g, device="cuda") * 3).to(getattr(torch, dtype))


def written(before, slots, keys, values, block):
    """The cache after a write, from the bytes before it."""
    cache = before.copy()
    dim = keys.shape[2]
    for t, slot in enumerate(slots):
        if not 0 <= slot < len(cache) * block:
            continue
        for which, x in enumerate((keys, values)):
            for h in range(x.shape[1]):
                pu.put_row(cache[slot // block, which, h], block, dim, slot % block, *pu.quantise(x[t, h], dim))
    return cache


def stands_for(cache, slots, block, dim):
    """float32 (keys, values) [tokens, heads, dim] of slots."""
    out = np.zeros((2, len(slots), cache.shape[2], dim), np.float32)
    for t, slot in enumerate(slots):
        if not 0 <= slot < len(cache) * block:
            continue
        for which in (0, 1):
            for h in range(cache.shape[2]):
                codes, pairs = pu.unpack(cache[slot // block, which, h], block, dim)
                out[which, t, h] = pu.value(codes[slot % block], pairs[slot % block], dim)
    return out


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("tokens,heads,dim,block", [
    (1, 1, 128, 16), (5, 3, 64, 1), (40, 2, 72, 100), (3, 5, 1, 4), (9, 1, 21, 3), (7, 2, 200, 16), (6, 1, 256, 32),
    (12, 4, 96, 7), (2, 2, 160, 5), (8, 1, 32, 2), (4, 1, 136, 16)])
def test_write_and_read(tok, tokens, heads, dim, block, dtype):
    import torch
    blocks = tokens // block + 3
    rng = np.random.default_rng(tokens * dim)
    before = rng.integers(0, 256, (blocks, 2, heads, pu.page_bytes(block, dim)), dtype=np.uint8)
    cache = torch.from_numpy(before).cuda()
    slots = rng.permutation(blocks * block)[:tokens]
    if tokens > 2:
        slots[1] = -1
    keys, values = rows((tokens, heads, dim), dtype), rows((tokens, heads, dim), dtype, 1)
    d_slots = torch.from_numpy(slots).cuda()
    tok.write_cache(cache, d_slots, keys, values, block)
    after = written(before, slots, keys.float().cpu().numpy(), values.float().cpu().numpy(), block)
    assert np.array_equal(cache.cpu().numpy(), after)  # every other byte as it was
    want = torch.from_numpy(stands_for(after, slots, block, dim))
    for out in (torch.float32, torch.float16, torch.bfloat16):
        k, v = tok.read_cache(cache, d_slots, dim, block, dtype=out)
        assert k.dtype is out and k.shape == keys.shape
        assert torch.equal(k.cpu(), want[0].to(out)) and torch.equal(v.cpu(), want[1].to(out))
    k, _ = tok.read_cache(cache, d_slots, dim, block)
    assert k.dtype is torch.float32
    # half a step of each group, and the roundings of its base and its largest element
    x = keys.double().cpu()
    for lo in range(0, dim, 32):
        g = x[..., lo:lo + 32]
        low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
        allowed = (high - low) / 30 * 1.01 + 2.0 ** -8 * (low.abs() + (high - low)) + 1e-30
        off = (k[..., lo:lo + 32].double().cpu() - g).abs()
        off[torch.from_numpy(slots) < 0] = 0
        assert bool((off <= allowed).all())


def test_values_at_the_ends_of_their_range(tok):
    """Equal elements, ranges below the step's smallest, the largest floats, zeros of both signs."""
    import torch
    big = 3.38e38
    cases = [np.full(64, 1.001), np.full(64, -7e37), np.zeros(64), np.linspace(-big, big, 64),
             np.linspace(1.0, 1.0 + 1e-7, 64), np.linspace(-1e-40, 1e-40, 64), np.linspace(0, 2.0 ** -98, 64),
             np.where(np.arange(64) % 2, -0.0, 0.0), np.linspace(-3e38, -2.9e38, 64), np.r_[np.zeros(63), 1.0],
             np.r_[np.full(63, 1e-30), 1e30], np.full(64, 2.0 ** -130)]
    x = np.array(cases, np.float32)[:, None, :]
    before = np.zeros((2, 2, 1, pu.page_bytes(8, 64)), np.uint8)
    cache = torch.from_numpy(before).cuda()
    slots = np.arange(len(x))
    d = torch.from_numpy(x).cuda()
    tok.write_cache(cache, torch.from_numpy(slots).cuda(), d, -d, 8)
    assert np.array_equal(cache.cpu().numpy(), written(before, slots, x, -x, 8))
    k, _ = tok.read_cache(cache, torch.from_numpy(slots).cuda(), 64, 8)
    assert bool(k.isfinite().all())
    span = np.ptp(x.astype(np.float64), -1)
    off = np.abs(k.cpu().numpy().astype(np.float64) - x).max(-1)
    assert np.all(off <= span / 30 * 1.01 + 2.0 ** -8 * (np.abs(x).max(-1).astype(np.float64) + span) + 2.0 ** -96)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3.4e38])
def test_a_spoiled_group_reads_back_as_nan(tok, bad):
    import torch
    x = rows((3, 2, 96), "float32")
    x[1, 0, 40] = bad
    cache = tok.new_cache(1, 4, 2, 96)
    slots = torch.tensor([2, 0, 3], device="cuda")
    tok.write_cache(cache, slots, x, x, 4)
    k, v = tok.read_cache(cache, slots, 96, 4)
    for y in (k, v):
        assert bool(y[1, 0, 32:64].isnan().all()) and int(y.isnan().sum()) == 32


def test_new_cache_stands_for_zeros(tok):
    import torch
    cache = tok.new_cache(5, 3, 2, 40)
    assert cache.shape == (5, 2, 2, pu.page_bytes(3, 40)) and cache.dtype is torch.uint8
    k, v = tok.read_cache(cache, torch.arange(15, device="cuda"), 40, 3)
    assert not bool(k.any()) and not bool(v.any())


def test_strides_layers_and_odd_addresses(tok):
    """A fused projection's keys and values, a layer among others in the blocks."""
    import torch
    heads, dim, block = 3, 64, 4
    fused = rows((10, 1, 2 * heads * dim + 5), "bfloat16")[:, 0]
    layers = torch.randint(0, 256, (6, 3, 2, heads, pu.page_bytes(block, dim)), dtype=torch.uint8, device="cuda")
    slots = torch.randperm(24, device="cuda")[:10]
    for start in (0, 1):
        keys = fused[:, start:start + heads * dim].unflatten(1, (heads, dim))
        values = fused[:, start + heads * dim:start + 2 * heads * dim].unflatten(1, (heads, dim))
        want = layers[:, 1].contiguous()
        others = layers[:, [0, 2]].clone()
        tok.write_cache(want, slots, keys.contiguous(), values.contiguous(), block)
        tok.write_cache(layers[:, 1], slots, keys, values, block)
        assert torch.equal(layers[:, 1], want) and torch.equal(layers[:, [0, 2]], others)
        for a, b in zip(tok.read_cache(layers[:, 1], slots, dim, block), tok.read_cache(want, slots, dim, block)):
            assert torch.equal(a, b)
    # one token for all slots, heads apart, elements apart
    one = rows((1, heads, dim), "float16")
    for x in (one.expand(10, heads, dim), one.transpose(0, 1).contiguous().transpose(0, 1).expand(10, heads, dim),
              rows((10, heads, 2 * dim), "float16")[..., ::2]):
        a, b = tok.new_cache(6, block, heads, dim), tok.new_cache(6, block, heads, dim)
        tok.write_cache(a, slots, x, x, block)
        tok.write_cache(b, slots, x.contiguous(), x.contiguous(), block)
        assert torch.equal(a, b)


def test_bad_slots_are_reported_and_left_out(bpe, tok):
    import torch
    x = rows((4, 1, 32), "float32")
    cache = tok.new_cache(2, 4, 1, 32)
    good = tok.new_cache(2, 4, 1, 32)
    status(bpe, tok)
    for bad in (8, -2, 2 ** 31, 2 ** 40, -2 ** 63):
        slots = torch.tensor([3, bad, -1, 6], device="cuda")
        tok.write_cache(cache, slots, x, x, 4)
        with pytest.raises(bpe.BpeError) as e:
            status(bpe, tok)
        assert e.value.code == 7
        tok.write_cache(good, slots[[0, 3]].contiguous(), x[[0, 3]], x[[0, 3]], 4)
        assert torch.equal(cache, good)
        k, _ = tok.read_cache(cache, slots, 32, 4)
        with pytest.raises(bpe.BpeError):
            status(bpe, tok)
        assert not bool(k[1:3].any()) and bool(k[[0, 3]].any())
    tok.write_cache(cache, torch.full((4,), -1, device="cuda"), x, x, 4)
    status(bpe, tok)
    assert torch.equal(cache, good)


def test_the_same_slot_twice_touches_no_other(tok):
    import torch
    x = rows((600, 2, 64), "float32")
    cache = tok.new_cache(4, 16, 2, 64)
    tok.write_cache(cache, torch.full((600,), 21, device="cuda"), x, x, 16)
    k, _ = tok.read_cache(cache, torch.arange(64, device="cuda"), 64, 16)
    assert bool(k[21].any()) and not bool(k[:21].any()) and not bool(k[22:].any())


def test_empty(tok):
    import torch
    cache, none = tok.new_cache(0, 4, 1, 32), torch.zeros(0, dtype=torch.int64, device="cuda")
    tok.write_cache(cache, none, torch.zeros(0, 1, 32, device="cuda"), torch.zeros(0, 1, 32, device="cuda"), 4)
    k, v = tok.read_cache(cache, none, 32, 4)
    assert k.shape == v.shape == (0, 1, 32)
    k, v = tok.read_cache(cache, torch.full((3,), -1, device="cuda"), 32, 4)
    assert not bool(k.any())


def test_a_cache_past_4_gigabytes(tok):
    import torch
    heads, dim, block = 8, 128, 256
    blocks = 6 * 2 ** 30 // (2 * heads * pu.page_bytes(block, dim))
    cache = torch.empty(blocks, 2, heads, pu.page_bytes(block, dim), dtype=torch.uint8, device="cuda")
    slots = torch.tensor([blocks * block - 1, 5, blocks * block - 300, (blocks * 2 // 3) * block + 17], device="cuda")
    x, y = rows((4, heads, dim), "float16"), rows((4, heads, dim), "float16", 2)
    tok.write_cache(cache, slots, x, y, block)
    small = tok.new_cache(1, block, heads, dim)
    tok.write_cache(small, torch.arange(4, device="cuda"), x, y, block)
    for a, b in zip(tok.read_cache(cache, slots, dim, block),
                    tok.read_cache(small, torch.arange(4, device="cuda"), dim, block)):
        assert torch.equal(a, b)


def test_refusals(bpe, tok):
    import torch
    x = torch.zeros(4, 2, 32, device="cuda")
    cache, slots = tok.new_cache(3, 4, 2, 32), torch.arange(4, device="cuda")
    for bad in (lambda: tok.write_cache(cache, slots, x.double(), x.double(), 4),
                lambda: tok.write_cache(cache, slots, x, x.half(), 4),
                lambda: tok.write_cache(cache, slots, x, x[:3], 4),
                lambda: tok.write_cache(cache, slots.int(), x, x, 4),
                lambda: tok.write_cache(cache, slots[:3], x, x, 4),
                lambda: tok.write_cache(cache, slots, x, x, 5),
                lambda: tok.write_cache(cache, slots, x[:, :1], x[:, :1], 4),
                lambda: tok.write_cache(cache[..., :-1], slots, x, x, 4),
                lambda: tok.write_cache(cache.transpose(1, 2), slots, x, x, 4),
                lambda: tok.write_cache(cache, slots, x.clone().requires_grad_(), x, 4),
                lambda: tok.read_cache(cache, slots, 64, 4),
                lambda: tok.read_cache(cache, slots, 32, 4, dtype=torch.float64),
                lambda: tok.read_cache(cache.float(), slots, 32, 4)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(bpe.BpeError):
        tok.new_cache(1, 4, 1, 257)
    with pytest.raises(bpe.BpeError):
        tok.new_cache(1, 0, 1, 32)
    wide = torch.zeros(3 * cache[0].numel() + 8, dtype=torch.uint8, device="cuda")
    odd = wide[8:].reshape(cache.shape)
    with pytest.raises(bpe.BpeError, match="16 bytes"):
        tok.write_cache(odd, slots, x, x, 4)
