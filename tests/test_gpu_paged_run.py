"""The operators on a paged cache together, as a server uses them: documents are
encoded, planned, embedded, their queries and keys turned, keys and values
written into their slots, attended to, and logits adjusted; then a token of each
request at a time, also as one captured graph that is replayed."""
import numpy as np
import pytest

from tests import paged_util as pu
from tests.ops_util import assert_close, byte_tokenizer, load

pytestmark = pytest.mark.gpu

HEADS, GROUP, DIM, BLOCK = 2, 2, 40, 8
ROWS = HEADS * GROUP


@pytest.fixture(scope="module")
def tok():
    t = byte_tokenizer(load())
    yield t
    t.close()


class Server:
    def __init__(self, tok, texts, n_new, dtype):
        import torch
        self.tok, self.n = tok, len(texts)
        g = torch.Generator(device="cuda")
        g.manual_seed(0)

        def weights(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") / shape[0] ** 0.5).to(dtype)

        self.embedding = weights(256, 64) * 16
        self.into, self.out = weights(64, (ROWS + 2 * HEADS) * DIM), weights(ROWS * DIM, 256)
        self.turns = tok.rotary_table(32)
        data = np.frombuffer(b"".join(texts), np.uint8).copy()
        offsets = np.cumsum([0] + [len(t) for t in texts]).astype(np.int64)
        self.ids, self.offsets = tok.encode(torch.from_numpy(data).cuda(), torch.from_numpy(offsets).cuda())
        width = -(-(max(len(t) for t in texts) + n_new) // BLOCK)
        self.table = torch.full((self.n, width), -1, dtype=torch.int32, device="cuda")
        blocks = self.n * width
        self.free = torch.randperm(blocks, device="cuda", generator=g).to(torch.int32)
        self.cache = tok.new_cache(blocks, BLOCK, HEADS, DIM)
        self.seq = self.head = None

    def step(self, ids, offsets, n_slots):
        """One step of new tokens: (logits of each request's last one, what attend took and gave)."""
        tok = self.tok
        self.seq, slots, positions, info = tok.plan_blocks(offsets, self.seq, self.table, self.free, BLOCK,
                                                           n_slots=n_slots, head=self.head)
        self.head = info[:1]
        x = tok.embed(ids, self.embedding)
        qkv = (x @ self.into).unflatten(1, (-1, DIM))
        turned = qkv[:, :ROWS + HEADS]
        tok.rotate(turned, positions, self.turns, out=turned)
        tok.write_cache(self.cache, slots, turned[:, ROWS:], qkv[:, ROWS + HEADS:], BLOCK)
        y = tok.attend(turned[:, :ROWS], self.cache, self.table, self.seq, BLOCK, offsets=offsets)
        last = y if offsets is None else y[offsets[1:] - 1]
        return last.flatten(1) @ self.out, (turned, qkv, slots, y)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_serving(tok, dtype):
    import torch

    import byte_level_bpe_pretokenize_gb300 as bpe
    texts = [b"the quick brown fox", b"x", b"jumps over the lazy dog, " * 9, b"ab"]
    n_new = 6
    s = Server(tok, texts, n_new, getattr(torch, dtype))
    new = [len(t) for t in texts]
    lens = np.zeros(len(texts), np.int64)
    ids, offsets = s.ids, s.offsets
    repetition = torch.full((s.n,), 1.3, device="cuda")
    output = torch.zeros(s.n, n_new, dtype=torch.int32, device="cuda")
    count = torch.zeros(s.n, dtype=torch.int32, device="cuda")
    for i in range(n_new):
        logits, (turned, qkv, slots, y) = s.step(ids, offsets, ids.numel())
        lens = lens + new
        assert s.seq.tolist() == lens.tolist()
        off = np.concatenate([[0], np.cumsum(new)])
        cache, table = s.cache.cpu().numpy(), s.table.cpu().numpy()
        want, bound = pu.attention(turned[:, :ROWS].double().cpu().numpy(), cache, table, lens, BLOCK, off,
                                   parts=2 if dtype == "float32" else 1)
        assert_close(y, torch.from_numpy(want), torch.from_numpy(bound), f"step {i}")
        # what is in the slots is what was quantised into them
        keys, values = tok.read_cache(s.cache, slots, DIM, BLOCK)
        for t in (0, ids.numel() - 1):
            for h in range(HEADS):
                for got, given in ((keys, turned[:, ROWS:]), (values, qkv[:, ROWS + HEADS:])):
                    row = pu.value(*pu.quantise(given[t, h].float().cpu().numpy(), DIM), DIM)
                    assert np.array_equal(got[t, h].cpu().numpy(), row)
        logits = tok.adjust_logits(logits, prompt=(s.ids, s.offsets), output=(output, count), repetition=repetition)
        ids = logits.argmax(1).to(torch.int32)
        output[:, i] = ids
        count += 1
        offsets, new = None, [1] * s.n
    bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)


def test_a_replayed_decode_step(tok):
    """The same requests served twice, eagerly and by replays of one captured step: equal tokens and caches."""
    import torch
    texts, n_new = [b"once there was", b"a", b" of the same kind as before" * 4], 10
    results = []
    for captured in (False, True):
        s = Server(tok, texts, n_new + 1, torch.bfloat16)
        logits, _ = s.step(s.ids, s.offsets, s.ids.numel())
        ids = logits.argmax(1).to(torch.int32)
        tokens = [ids.clone()]
        if captured:
            seq, head = s.seq.clone(), s.head.clone()
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                s.seq, s.head = seq, head
                logits, _ = s.step(ids, None, s.n)
                ids.copy_(logits.argmax(1))
                seq.copy_(s.seq)
                head.copy_(s.head)
            for _ in range(n_new):
                graph.replay()
                tokens.append(ids.clone())
        else:
            for _ in range(n_new):
                logits, _ = s.step(ids, None, s.n)
                ids = logits.argmax(1).to(torch.int32)
                tokens.append(ids.clone())
        results.append((torch.stack(tokens), s.cache, s.table))
    for a, b in zip(*results):
        assert torch.equal(a, b)
