"""Windows that cut the cache of many units in the split form: units that lie in several runs are joined, whatever the
lengths, and every row is written."""
import pytest
import torch

import pyramid_top_block_gb300 as pisa
from test_gpu_cache import DEV, gen, i32, make_cache, normal, status
from test_gpu_cache_scores import check, expected, slopes_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("cap,slopes", [(0.0, False), (0.0, True), (30.0, False), (30.0, True)])
@pytest.mark.parametrize("B,T,G,Hkv,page,lengths,window", [
    (32, 1, 4, 2, 64, [16421] * 32, 4096),
    (24, 1, 2, 2, 16, [(b * 977) % 9000 for b in range(24)], 4000),      # some shorter than the window, one empty
    (8, 1, 2, 8, 32, [5000, 20000, 1, 64, 4096, 4097, 12345, 8191], 4200),
    (5, 5, 16, 2, 64, [9000, 4, 30000, 7001, 7000], 7000),               # five row tiles of each
    (40, 3, 1, 1, 128, [6000 + 400 * b for b in range(40)], 6001),
])
def test_windows_of_many_units(bits, cap, slopes, B, T, G, Hkv, page, lengths, window):
    g = gen(B * T + page)
    Hq = G * Hkv
    cache = make_cache(g, B, max(lengths) + 9, Hkv, page, bits)
    q, s = normal(g, B, T, Hq, 64) * (3.0 if cap else 1.0), slopes_of(Hq) if slopes else None
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((B, T, Hq, 64), 7.0, dtype=dtype, device=DEV)
        ws = pisa.cache_workspace(cache)
        pisa.cache_attention(q, cache, i32(lengths), out=out, workspace=ws, cap=cap, slopes=s, window=window)
        assert status(ws) == 0
        check(out, expected(q, cache, lengths, window, cap, s, dtype))


def test_a_window_does_not_depend_on_the_other_sequences():
    """A sequence's rows are the same beside others, whose runs lie elsewhere, up to the order of the sums."""
    g = gen(6)
    lengths, window = [30000, 16384, 5000, 100] * 10, 4500
    cache = make_cache(g, 40, 30000, 2, 64, 16)
    q = normal(g, 40, 1, 8, 64)
    out = pisa.cache_attention(q, cache, i32(lengths), window=window)
    for b in (0, 1, 2, 3, 17, 38):
        one = pisa.PagedCache(cache.pages, cache.table[b:b + 1].contiguous(), 64)
        alone = pisa.cache_attention(q[b:b + 1].contiguous(), one, i32(lengths[b:b + 1]), window=window)
        assert bool(((out[b:b + 1].float() - alone.float()).abs() <= 2.0 ** -7 * alone.float().abs().amax()).all())
