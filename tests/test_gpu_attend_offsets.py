"""Offsets that fall: requests that share tokens, among them so many that long
runs have more columns than the tokens could have."""
import numpy as np
import pytest

from tests import paged_close as pc
from tests.ops_util import ROUNDOFF, byte_tokenizer, load
from tests.test_gpu_attend import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,group,dim", [(16, 1, 64), (4, 4, 96), (8, 8, 32)])
def test_long_runs_that_share_tokens(heads, group, dim):
    import torch
    bpe = load()
    tok = byte_tokenizer(bpe)
    n = 2000
    # requests 0, 2 and 3 have tokens [0, 1000), [0, 1000) and [1000, 2000); request 1 falls
    b = Batch([1000, 1000, 1000, 1100], heads, group, dim, 16, new=[500] * 4, seed=1)
    offsets = np.array([0, 1000, 0, 1000, 2000])
    out = torch.full((n, heads * group, dim), 9.0, dtype=b.q.dtype, device="cuda")
    got = b.run(tok, offsets=torch.from_numpy(offsets).cuda(), out=out).double().cpu().numpy()
    with pytest.raises(bpe.BpeError) as e:
        bpe.bpe_sync_status(tok.handle, torch.cuda.current_stream().cuda_stream)
    assert e.value.code == 7
    q = b.q.double().numpy()
    near = []
    for r in (0, 2, 3):
        rows = slice(offsets[r], offsets[r] + 1000)
        want, bound = pc.attention(q[rows], b.cache, b.table[r:r + 1], b.lens[r:r + 1], 16, [0, 1000])
        u = ROUNDOFF["bfloat16"]
        near.append(np.abs(got[rows] - want) <= bound + u * (np.abs(want) + bound))
    assert near[2].all()  # tokens of one request alone
    # each element of the shared ones is one of the two requests'
    assert (near[0] | near[1]).all()
    tok.close()
