"""What the example generates for a request does not depend on the batch around
it: every request alone, in pairs and all together. The model's numbers are
small whole ones, so that logits are exact in any order of summation."""
import pytest

from tests.test_gpu_example import example  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("masked", [False, True])
def test_requests_alone(example, masked):  # noqa: F811
    import torch

    import workloads
    merges, vb, vo = workloads.table(1)
    tok = example.bpe.Tokenizer(merges, vb, vo)
    model = example.Model(tok, dim=64)  # a scale of 8; states are multiples of 2 below 1400, their products exact in f32
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    with torch.no_grad():
        for table in (model.table, model.out):
            table.copy_(torch.randint(-100, 101, table.shape, generator=g, device="cuda"))
    allowed = example.letters_and_spaces(vb, vo) if masked else None
    prompts = [b"the", b"x" * 40, b"what is", b" of the same kind as before,", b"a"]
    together = model.generate(prompts, 20, allowed)
    assert len(set(together)) > 1
    assert [model.generate([p], 20, allowed)[0] for p in prompts] == together
    assert model.generate(prompts[3:], 20, allowed) == together[3:]
    assert model.generate(prompts[::-1], 20, allowed) == together[::-1]
    tok.close()
