"""A small language model around the tokenizer, on one GPU: trained on encoded
documents, then served with a paged cache, penalties and a grammar mask.

The state after a token is a decaying sum of the embeddings of the last few
tokens, and the logits of the next token are the state times an output table.

    train   encode -> embed -> states -> logits -> loss -> embed_grad -> update
    serve   encode -> plan_blocks -> embed -> cache -> states -> logits
            -> adjust_logits -> the best token -> plan_blocks -> ... -> decode

Run: python examples/small_lm.py
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import byte_level_bpe_pretokenize_gb300 as bpe  # noqa: E402
import workloads  # noqa: E402

BLOCK = 16           # cache slots of a block
DECAY = (1.0, 0.5, 0.25)  # weight of the last token, the one before it, ...


def device(array):
    return torch.from_numpy(np.array(array)).cuda()


def owners(offsets, total):
    """The document of each of `total` packed tokens."""
    return torch.searchsorted(offsets, torch.arange(total, device="cuda"), right=True) - 1


class Model:
    def __init__(self, tok: bpe.Tokenizer, dim: int = 128, seed: int = 0):
        self.tok, self.dim = tok, dim
        self.vocab = bpe.bpe_table_info(tok.handle)[1]
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.table = (torch.randn(self.vocab, dim, generator=gen, device="cuda") / dim).requires_grad_()
        self.out = torch.zeros(self.vocab, dim, device="cuda", requires_grad=True)
        self.scale = dim ** 0.5

    # ------------------------------------------------------------- training --

    def step(self, data, offsets, rate: float) -> float:
        """One step on documents (uint8, int64 offsets, on the GPU): the loss
        of every token of every document given those before it."""
        ids, offs = self.tok.encode(data, offsets)
        n = ids.numel()
        x = self.tok.embed(ids, self.table, scale=self.scale)  # its backward pass is embed_grad
        place = torch.arange(n, device="cuda") - offs[owners(offs, n)]
        state = sum(w * torch.where((place >= k)[:, None], x.roll(k, 0), 0.0) for k, w in enumerate(DECAY))
        follows = place[1:] > 0  # the next token is of the same document
        logits = state[:-1][follows] @ self.out.t()
        loss = torch.nn.functional.cross_entropy(logits, ids[1:][follows].long())
        self.table.grad = self.out.grad = None
        loss.backward()
        with torch.no_grad():
            for p in (self.table, self.out):
                p -= rate * p.grad
        return float(loss.detach())

    # -------------------------------------------------------------- serving --

    @torch.no_grad()
    def generate(self, prompts: list[bytes], n_new: int, allowed: torch.Tensor | None = None):
        """Greedy continuations (bytes) of prompts. allowed: bool[vocab], the
        tokens that may be chosen."""
        tok, n = self.tok, len(prompts)
        blob, ends = b"".join(prompts), np.cumsum([0] + [len(p) for p in prompts])
        ids, offs = tok.encode(device(np.frombuffer(blob, np.uint8)), device(ends.astype(np.int64)))
        longest = max(len(p) for p in prompts) + n_new  # no prompt has more tokens than bytes
        width = -(-longest // BLOCK)
        table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
        free = torch.randperm(n * width, device="cuda").to(torch.int32)
        cache = torch.zeros(n * width * BLOCK, self.dim, device="cuda")
        output = torch.zeros(n, n_new, dtype=torch.int32, device="cuda")
        lens = torch.zeros(n, dtype=torch.int32, device="cuda")
        repetition = torch.full((n,), 1.2, device="cuda")
        frequency = torch.full((n,), 0.4, device="cuda")
        mask = None
        if allowed is not None:
            bits = torch.zeros((self.vocab + 31) // 32 * 32, dtype=torch.int64, device="cuda")
            bits[:self.vocab] = allowed
            mask = (bits.reshape(-1, 32) << torch.arange(32, device="cuda")).sum(1).to(torch.int32)[None].contiguous()
            rows = torch.zeros(n, dtype=torch.int32, device="cuda")

        # the prompts, then a token of each request at a time; nothing waits for the host
        new_ids = ids
        seq, slots, _, info = tok.plan_blocks(offs, None, table, free, BLOCK, n_slots=ids.numel())
        for step in range(n_new):
            cache[slots] = tok.embed(new_ids, self.table, scale=self.scale)
            state = torch.zeros(n, self.dim, device="cuda")
            for k, w in enumerate(DECAY):
                at = (seq.long() - 1 - k).clamp(min=0)
                slot = table.gather(1, (at // BLOCK)[:, None])[:, 0].long() * BLOCK + at % BLOCK
                state += w * torch.where((seq > k)[:, None], cache[slot.clamp(min=0)], 0.0)
            logits = tok.adjust_logits(state @ self.out.t(), prompt=(ids, offs), output=(output, lens),
                                       repetition=repetition, frequency=frequency, mask=mask,
                                       mask_rows=None if mask is None else rows)
            new_ids = logits.argmax(1).to(torch.int32)
            output[:, step] = new_ids
            lens += 1
            seq, slots, _, info = tok.plan_blocks(None, seq, table, free, BLOCK, head=info[:1])
        bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)
        text, text_offs = tok.decode(output.reshape(-1), torch.arange(n + 1, device="cuda") * n_new)
        text, text_offs = bytes(text.cpu().numpy()), text_offs.tolist()
        return [text[a:b] for a, b in zip(text_offs, text_offs[1:])]


def letters_and_spaces(vocab_bytes, vocab_offsets) -> torch.Tensor:
    """The tokens of lower-case letters and spaces alone."""
    allowed = np.zeros(len(vocab_offsets) - 1, dtype=bool)
    good = set(b"abcdefghijklmnopqrstuvwxyz ")
    for t in range(len(allowed)):
        token = bytes(vocab_bytes[vocab_offsets[t]:vocab_offsets[t + 1]])
        allowed[t] = len(token) > 0 and set(token) <= good
    return device(allowed)


def main(steps: int = 60, docs: int = 64, n_new: int = 24):
    merges, vb, vo = workloads.table(1)
    tok = bpe.Tokenizer(merges, vb, vo)
    model = Model(tok)
    losses = []
    for step in range(steps):
        data, offsets = workloads.docs(1, (step * docs) % 192, docs)
        losses.append(model.step(device(data), device(offsets), rate=1.0))
        if step % 10 == 0 or step == steps - 1:
            print(f"step {step:3d}  loss {losses[-1]:.3f}")
    prompts = [b"the", b"Once there was", b"a", b" of the same kind as before,"]
    texts = model.generate(prompts, n_new, letters_and_spaces(vb, vo))
    for p, t in zip(prompts, texts):
        print(repr(p), "->", repr(t))
    tok.close()
    return losses, prompts, texts


if __name__ == "__main__":
    main()
