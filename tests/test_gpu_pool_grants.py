"""Grants written in the counts' own place."""
import random

import pytest
import torch

import pyramid_top_block_gb300 as pisa
from test_gpu_cache import i32
from test_gpu_pool import make_pool, mirror, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,n_pages", [(40, 200), (40, 90), (300, 6000), (300, 500)])
def test_grants_in_place_of_the_counts(B, n_pages):
    """One CTA and a cluster, with enough pages and too few."""
    r = random.Random(B + n_pages)
    wide, page, T = 20, 16, 40
    held = [r.randrange(0, max(1, min(wide - 4, n_pages // (2 * B))) + 1) for _ in range(B)]
    pages, table, refs, lengths = make_pool(r, B, wide, n_pages, page, held)
    m = mirror(pages, table, refs, lengths, page)
    counts = [r.choice([0, T, T + 7, -2, r.randint(0, T)]) for _ in range(B)]
    granted, bad = m.reserve([min(max(c, 0), T) for c in counts])
    assert not bad
    x = i32(counts)
    got = pisa.cache_reserve(pisa.PagePool(pages, table, refs, page), lengths, T, counts=x, granted=x)
    assert got is x and x.tolist() == granted
    same(m, pages, table, refs, lengths)


def test_lists_that_lie_in_one_another_are_refused():
    r = random.Random(1)
    pages, table, refs, lengths = make_pool(r, 8, 4, 40, 16, [2] * 8)
    pool = pisa.PagePool(pages, table, refs, 16)
    both = torch.zeros(9, dtype=torch.int32, device=pages.device)
    for kw in (dict(granted=lengths), dict(counts=both[:8], granted=both[1:])):
        with pytest.raises(pisa.PisaError):
            pisa.cache_reserve(pool, lengths, 3, **kw)
    with pytest.raises(pisa.PisaError):
        pisa.cache_fork(pool, lengths, lengths)
    with pytest.raises(pisa.PisaError):
        pisa.cache_compact(pool, used=refs[:1])
