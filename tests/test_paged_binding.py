"""Checks of the paged binding's plain arguments, without a GPU."""
import pytest
import torch

import kv_cache_compression_fkv_b200 as fkv


@pytest.mark.parametrize("kw", [{"window": 2 ** 31}, {"window": 2 ** 32 + 5}, {"window": -1}, {"num_q_heads": 2 ** 32 + 4},
                                {"num_q_heads": 0}])
def test_sizes_beyond_32_bits_are_refused(kw):
    """A C int would take 2^32 + 5 as 5, without a word."""
    k = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16)
    t = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError, match=next(iter(kw))):
        fkv.PagedCache(k, k, t, **{"num_q_heads": 4, **kw})


@pytest.mark.parametrize("pairs", [(2 ** 32 + 4, -2 ** 32), (-1, 5)])
def test_axis_pairs_out_of_range_are_refused(pairs):
    with pytest.raises(ValueError, match="axis_pairs"):
        fkv.make_rope(torch.zeros(4), axis_pairs=pairs)
