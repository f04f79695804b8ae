"""Scales that are no finite number once they are powers of two are refused by the
library before it touches the GPU."""
import ctypes

import pytest


@pytest.mark.parametrize("scale,ok", [(0.125, True), (-0.125, True), (0.0, True), (2.3e38, True), (2.4e38, False),
                                      (-3.3e38, False), (float("inf"), False), (float("nan"), False)])
def test_scales(scale, ok):
    import torch

    import __graft_entry__
    __graft_entry__.build()
    import byte_level_bpe_pretokenize_gb300 as bpe
    if torch.cuda.is_available():
        pytest.skip("the pointers here are no device pointers")
    handle, base = ctypes.create_string_buffer(1 << 16), 1 << 20
    a = bpe.AttendArgs(queries=base, out=2 * base, query_token_stride=32, query_head_stride=32, out_token_stride=32,
                       out_head_stride=32, n_tokens=1, n_heads=1, group=1, dim=32, cache=base, n_blocks=1,
                       block_stride=base, block_size=16, table=base, max_blocks=1, table_stride=1, seq_lens=base,
                       n_requests=1, scale=scale)
    with pytest.raises(bpe.BpeError) as e:  # without a GPU any call ends with an error
        bpe.bpe_attend(ctypes.addressof(handle), a, 0)
    assert (e.value.code == 1 and "scale" in str(e.value)) is not ok
