"""Forked sequences of layers that select: pages are shared, and the caller copies the pyramid's rows, as documented."""
import pytest
import torch

import pyramid_top_block_gb300 as pisa
from test_gpu_cache import DEV, check_attention, gen, i32, normal, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [16, 4])
def test_samples_of_a_prompt_select_from_its_history(bits):
    g = gen(bits)
    B, N, cap, Hq, Hkv, K = 4, 1500, 1700, 16, 2, 8
    pool = pisa.PagePool.allocate(B, cap, Hkv, n_pages=120, page_size=64, bits=bits)
    cache, pws, ws = pool.layer(), pisa.pool_workspace(pool), pisa.cache_workspace(pool.layer())
    pyr = pisa.Pyramid.allocate(torch.zeros(B, cap, Hkv, 64, dtype=torch.bfloat16, device=DEV), with_lengths=True)
    rotary = pisa.rotary_table(cap)
    # two prompts, of 1500 tokens and of 700, in sequences 0 and 2
    counts = i32([N, 0, 700, 0])
    n = pisa.cache_reserve(pool, pyr.lengths, N, counts=counts, workspace=pws)
    assert n.tolist() == [N, 0, 700, 0]
    q, k, v = normal(g, B, N, Hq, 64), normal(g, B, N, Hkv, 64), normal(g, B, N, Hkv, 64)
    pisa.cache_append(q, k, v, cache, pyr.lengths, rotary, counts=n, k_out=pyr.keys[:, :N], workspace=ws)
    pyr.lengths += n
    pisa.build_pyramid_ragged(pyr)
    # 1 becomes a sample of 0, and 3 of 2
    parents = i32([0, 0, 2, 2])
    pisa.cache_fork(pool, parents, pyr.lengths, workspace=pws)
    for x in (pyr.keys, pyr.summaries):
        x.copy_(x[parents.long()])
    assert pyr.lengths.tolist() == [N, N, 700, 700]
    for step in range(70):  # past a block's end: leaves and pages of their own
        same = step == 0
        q, k, v = normal(g, B, 1, Hq, 64), normal(g, B, 1, Hkv, 64), normal(g, B, 1, Hkv, 64)
        if same:
            q, k, v = (x[parents.long()].contiguous() for x in (q, k, v))
        n = pisa.cache_reserve(pool, pyr.lengths, 1, workspace=pws)
        assert n.tolist() == [1] * B
        q, k = pisa.cache_append(q, k, v, cache, pyr.lengths, rotary, counts=n, workspace=ws)
        idx, _ = pisa.decode_append_and_select(q[:, 0], k[:, 0], pyr, K)
        out = pisa.cache_attention(q, cache, pyr.lengths, idx=idx, workspace=ws)
        if same:
            assert torch.equal(idx[1], idx[0]) and torch.equal(idx[3], idx[2])
            assert torch.equal(out[1], out[0]) and torch.equal(out[3], out[2])
        lengths = pyr.lengths.tolist()
        if step % 23 == 0:
            check_attention(cache, q, lengths, out, idx=idx[:, :, None])
    assert status(ws) == 0 and status(pws) == 0
    # the selection is that of pyramids built anew over the same keys
    fresh = pisa.Pyramid.allocate(pyr.keys.clone(), with_lengths=True)
    fresh.lengths.copy_(pyr.lengths)
    pisa.build_pyramid_ragged(fresh)
    q, k = normal(g, B, Hq, 64), normal(g, B, Hkv, 64)
    a, _ = pisa.decode_append_and_select(q, k, pyr, K)
    b, _ = pisa.decode_append_and_select(q, k, fresh, K)
    assert torch.equal(a, b)
