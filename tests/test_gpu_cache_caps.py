"""Caps that a C float does not hold are refused like others out of range."""
import pytest
import torch

import pyramid_top_block_gb300 as pisa
from test_gpu_cache import gen, i32, make_cache, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap", [1e-46, -1e-46, 1e-300, -1e-300, 1e39, -1e39, 1e300])
def test_caps_past_the_range_of_floats(cap):
    g = gen(1)
    cache = make_cache(g, 1, 40, 1, 16, 16)
    q, n = normal(g, 1, 2, 4, 64), i32([30])
    with pytest.raises(pisa.PisaError):
        pisa.cache_attention(q, cache, n, cap=cap)
    with pytest.raises(pisa.PisaError):
        pisa.cache_prompt_attention(q, cache, n, cap=cap)
    plain = pisa.cache_attention(q, cache, n)
    assert torch.equal(pisa.cache_attention(q, cache, n, cap=-0.0), plain)
