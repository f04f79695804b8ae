"""The example runs the tokenizer and the operators around the model together:
its loss falls, its gradient is the one of plain torch, and what it generates
follows the mask and does not depend on the batch around a request."""
import pytest

from tests.ops_util import load

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    load()
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "small_lm.py")
    spec = importlib.util.spec_from_file_location("small_lm", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_main(example):
    losses, prompts, texts = example.main(steps=30)
    assert losses[-1] < losses[0] - 0.5
    assert len(texts) == len(prompts)
    for t in texts:
        assert len(t) >= 24 and set(t) <= set(b"abcdefghijklmnopqrstuvwxyz ")


def test_step_is_plain_torch(example):
    """One training step against the same step with torch's own indexing."""
    import torch

    import workloads
    tok = example.bpe.Tokenizer(*workloads.table(1))
    data, offsets = (example.device(x) for x in workloads.docs(1, 0, 8))
    a, b = example.Model(tok), example.Model(tok)

    class Plain:
        encode = tok.encode

        @staticmethod
        def embed(ids, weight, scale):
            return weight[ids.long()] * scale

    b.tok = Plain
    losses = a.step(data, offsets, 0.5), b.step(data, offsets, 0.5)
    assert abs(losses[0] - losses[1]) <= 1e-5 * abs(losses[1])
    # the two add a row's gradients in another order: 1e-5 of the largest is far above that
    assert float((a.table.grad - b.table.grad).abs().max()) <= 1e-5 * float(b.table.grad.abs().max())
    tok.close()


def test_generation_repeats(example):
    """The free list is dealt in another order each time; what is generated is the same."""
    import workloads
    merges, vb, vo = workloads.table(1)
    tok = example.bpe.Tokenizer(merges, vb, vo)
    model = example.Model(tok, seed=3)
    data, offsets = (example.device(x) for x in workloads.docs(1, 0, 16))
    model.step(data, offsets, 1.0)
    prompts = [b"the", b"x" * 40, b"what is"]
    together = model.generate(prompts, 20)
    assert together == model.generate(prompts, 20)
    tok.close()
