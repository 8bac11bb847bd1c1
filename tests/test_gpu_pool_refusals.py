"""Numbers that the C ABI's 32 bits would cut."""
import pytest
import torch

import pyramid_top_block_gb300 as pisa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1 << 31, (1 << 32) + 1, -(1 << 32) + 1])
def test_reserves_of_more_tokens_than_32_bits_hold(T):
    pool = pisa.PagePool.allocate(2, 100, 1, 10, page_size=16)
    lengths = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="32 bits"):
        pisa.cache_reserve(pool, lengths, T)
    assert not bool(pool.refs.any()) and bool((pool.table == -1).all())
