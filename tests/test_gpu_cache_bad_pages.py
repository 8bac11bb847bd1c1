"""A page number out of range reaches the queries that see one of its tokens, and no others."""
import pytest
import torch

import pyramid_top_block_gb300 as pisa
import test_gpu_cache as base

pytestmark = pytest.mark.gpu
DEV = base.DEV


def check(cache, good, q, lengths, first_bad, idx=None):
    """Queries that see token first_bad[b] of their sequence, or a later one, are NaN; the others are as over `good`."""
    T = q.shape[1]
    ws = pisa.cache_workspace(cache)
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
        pisa.cache_attention(q, cache, base.i32(lengths), idx=idx, out=out, workspace=ws)
        assert base.status(ws) == 6
        sees = {(b, t): lengths[b] - T + t + 1 > first_bad[b] for b in range(len(lengths)) for t in range(T)}
        assert any(sees.values()) and not all(sees.values())
        for (b, t), bad in sees.items():
            assert bool(torch.isnan(out[b, t]).all()) == bad, (b, t)
            assert bad or not bool(torch.isnan(out[b, t]).any()), (b, t)
        rows = {k for k, bad in sees.items() if not bad}
        base.check_attention(good, q, lengths, out, idx=idx, rows=rows)


@pytest.mark.parametrize("bad", [-1, 1 << 30])
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("T,G,page,lengths", [
    (4, 4, 16, [130, 127]),    # queries 2 and 3 of the first sequence see the last page; all of the second see none of it
    (2, 16, 64, [65, 64]),
    (16, 1, 32, [1034, 7]),    # a sequence shorter than T: its first queries see nothing
    (5, 8, 128, [1283, 1280]),
    (7, 2, 16, [3, 40]),
])
def test_only_queries_that_see_a_bad_page(bad, bits, T, G, page, lengths):
    g = base.gen(T * 100 + page)
    good = base.make_cache(g, 2, 1400, 2, page, bits)
    q = base.normal(g, 2, T, 2 * G, 64)
    table = good.table.clone()
    first_bad = []
    for b, n in enumerate(lengths):  # the page of the first sequence's newest token, and the same page of the other
        at = (lengths[0] - 1) // page
        table[b, at] = bad
        first_bad.append(at * page)
    cache = pisa.PagedCache(good.pages, table, page)
    check(cache, good, q, lengths, first_bad)
    check(base.in_a_wide_table(cache), good, q, lengths, first_bad)
    blocks = -(-max(lengths) // 64)
    idx = torch.randperm(blocks, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(DEV)
    idx = idx.expand(2, 2, T, blocks).contiguous()
    check(cache, good, q, lengths, first_bad, idx=idx)


@pytest.mark.parametrize("bits", [16, 4])
def test_a_bad_page_in_a_long_cache(bits):
    """Units in several runs, several row tiles a unit."""
    g = base.gen(5)
    T, G, page = 9, 16, 64
    lengths = [9030, 9024]
    good = base.make_cache(g, 2, 9100, 2, page, bits)
    table = good.table.clone()
    table[:, 141] = good.n_pages  # tokens 9024 ..: queries 3 .. 8 of the first sequence see it, none of the second
    cache = pisa.PagedCache(good.pages, table, page)
    check(cache, good, base.normal(g, 2, T, 2 * G, 64), lengths, [9024, 9024])
