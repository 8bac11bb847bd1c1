"""What a query does not see does not change a bit of its result, capped and biased scores among them."""
import pytest
import torch

import cache_ref as ref
import pyramid_top_block_gb300 as pisa
from test_gpu_cache import DEV, gen, i32, make_cache, normal

pytestmark = pytest.mark.gpu


def scaled_keys(cache, positions, factor):
    """Keys of a sequence's positions times a power of two (4 bits: their scales' exponents)."""
    U, P = min(cache.page_size, 64), cache.page_size
    for p in positions:
        page, rec, u = int(cache.table[0, p // P]), (p % P) // U, p % U
        if cache.bits == 16:
            cache.pages[page, :, rec, 0, u] *= 2.0 ** factor
        else:
            cache.pages[page, :, rec, 32 * U + 4 * u:32 * U + 4 * u + 4] += 8 * factor


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("cap,slopes", [(0.0, False), (6.0, False), (40.0, True), (300.0, False), (0.0, True)])
@pytest.mark.parametrize("window,start,T", [(0, 100, 300), (50, 300, 200), (0, 5000, 20)])
def test_unseen_keys_do_not_choose_how_scores_are_computed(bits, cap, slopes, window, start, T):
    """Scores that are seen stay below half the cap; those behind the sequence and before the windows may pass it."""
    g = gen(bits + T)
    n = start + T
    cache = make_cache(g, 1, n + 100, 2, 64, bits)
    q = normal(g, 1, T, 32, 64)
    if cap:  # the largest seen score is a third of the cap
        k, _ = ref.tokens(cache, 0, n)
        q = (q * (cap / 3 / float((q[0, :, 0].double() @ k[:, 0].T / 8).abs().max()) / 1.5)).to(torch.bfloat16)
    s = torch.tensor([2.0 ** (-8 * (h + 1) / 32) for h in range(32)], device=DEV) if slopes else None
    unseen = list(range(n, n + 100)) + list(range(max(0, start + 1 - window) if window else 0))
    outs = []
    for factor in (0, 4, 2):
        scaled_keys(cache, unseen[:160], factor)
        for call in (lambda: pisa.cache_prompt_attention(q, cache, i32([start]), cap=cap, slopes=s, window=window),
                     lambda: pisa.cache_attention(q[:, -5:], cache, i32([n]), cap=cap, slopes=s, window=window),
                     lambda: pisa.cache_attention(q[:, -5:], cache, i32([n]), cap=cap, slopes=s, window=window,
                                                  out=torch.empty(1, 5, 32, 64, device=DEV))):
            outs.append(call())
    for a, b in zip(outs[3:], outs[:3] * 2):
        assert torch.equal(a, b), float((a.float() - b.float()).abs().max())
