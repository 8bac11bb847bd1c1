"""What the attention calls ask for of a workspace: the single tokens' call no more than its partial results take."""
import pytest
import torch

import pyramid_top_block_gb300 as pisa
from test_cache_abi import attend, cache
from test_more_cache_abi import prompt, scored


def test_a_decoding_programs_workspace():
    lib = pisa.load()
    token, every = lib.pisa_cache_attention_workspace_bytes(), lib.pisa_cache_workspace_bytes()
    # two partial results (16 rows of 64 sums, a reference and a sum of weights) for each of 152 CTAs, and the status
    assert token == 256 + 152 * 2 * 16 * 66 * 4 < every
    assert pisa.cache_workspace_bytes(prompts=False) == token and pisa.cache_workspace_bytes() == every
    assert attend(cache(), ws_bytes=token - 1) == 3 and scored(cache(), ws_bytes=token - 1) == 3
    assert prompt(cache(), ws_bytes=token) == 3 and prompt(cache(), ws_bytes=every - 1) == 3


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [16, 4])
def test_calls_keep_within_it(bits):
    """The split form with many cut units and several row tiles, the workspace's end followed by a mark."""
    from test_gpu_cache import DEV, gen, i32, make_cache, normal, status
    g = gen(bits)
    lengths = [9000, 20000, 31, 12000, 7777, 15000]
    c = make_cache(g, 6, 20000, 2, 64, bits)
    q, n = normal(g, 6, 5, 32, 64), i32(lengths)
    need = pisa.cache_workspace_bytes(prompts=False)
    room = torch.zeros(need + 4096, dtype=torch.uint8, device=DEV)
    room[need:] = 0xa5
    for kw in (dict(), dict(window=5000), dict(cap=20.0), dict(slopes=torch.rand(32, device=DEV))):
        want = pisa.cache_attention(q, c, n, **kw)  # scratch of its own
        assert torch.equal(pisa.cache_attention(q, c, n, workspace=room[:need], **kw), want)
        assert torch.equal(pisa.cache_attention(q, c, n, workspace=pisa.cache_workspace(c), **kw), want)
    assert status(room[:need]) == 0 and bool((room[need:] == 0xa5).all())
    with pytest.raises(pisa.PisaError):
        pisa.cache_prompt_attention(q, c, n - 5, workspace=pisa.cache_workspace(c, prompts=False))
