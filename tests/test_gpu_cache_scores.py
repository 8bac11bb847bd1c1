"""Attention of the newest tokens with a window, capped scores or a bias by distance, against 64 bits."""
import pytest
import torch

import cache_ref as ref
import pyramid_top_block_gb300 as pisa
import score_ref
from test_gpu_cache import DEV, gen, i32, make_cache, normal, status

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def slopes_of(Hq):
    return torch.tensor([2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)], device=DEV)


def expected(q, cache, lengths, window, cap, slopes, dtype, idx=None):
    """(o, tolerance) float64 [B, T, Hq, 64] of cache_attention."""
    B, T, Hq, _ = q.shape
    o, tol = torch.zeros(B, T, Hq, 64, dtype=torch.float64, device=DEV), torch.zeros(B, T, Hq, 64, dtype=torch.float64, device=DEV)
    weight = {(16, torch.bfloat16): 2.0 ** -16, (16, torch.float32): 2.0 ** -22, (4, torch.bfloat16): 2.0 ** -11,
              (4, torch.float32): 2.0 ** -20}[cache.bits, dtype]
    for b in range(B):
        n = int(lengths[b])
        if n == 0:
            continue
        k, v = ref.tokens(cache, b, n)
        at = n - T + torch.arange(T, device=DEV)
        lo = (at - window + 1).clamp(min=0) if window else torch.zeros_like(at)
        x, pv, big = score_ref.attention(q[b].double(), k, v, at, lo, at + 1, cap, slopes)
        o[b] = x
        tol[b] = score_ref.tolerance(x, pv, big, n, weight, dtype, cap)
        if cache.bits == 4:  # fp16 weights' steps of 2^-35 of the largest weight at least
            seen_v = v.abs().sum(0)  # [Hkv, 64]
            tol[b] += 2.0 ** -35 * seen_v.repeat_interleave(Hq // cache.Hkv, 0)
    return o, tol


def check(got, want):
    o, tol = want
    off = (got.double() - o).abs()
    assert bool((off <= tol).all()), float((off / tol).max())


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("B,T,G,Hkv,page,lengths,window,cap,slopes,scale", [
    (2, 3, 8, 2, 64, [20000, 300], 0, 0.0, True, 1.0),
    (1, 2, 4, 1, 32, [5000], 0, 0.0, True, 2.0 ** -70),       # queries so small that the bias alone decides
    (1, 2, 4, 1, 32, [500], 0, 500.0, True, 3.0),             # a cap taken by the polynomial
    (1, 1, 1, 1, 16, [1], 0, 5.0, True, 3.0),
    (2, 1, 16, 2, 64, [300, 0], 0, 2.0, False, 4.0),          # scores past the cap
    (3, 1, 8, 2, 64, [4097, 65, 64], 64, 0.0, False, 1.0),
    (2, 3, 4, 2, 32, [700, 2], 100, 30.0, True, 3.0),
    (2, 16, 16, 1, 128, [515, 16], 7, 0.0, False, 1.0),       # windows shorter than the queries are apart
    (2, 16, 1, 3, 16, [130, 33], 1, 50.0, True, 3.0),         # each query sees itself alone
    (1, 5, 2, 2, 256, [9000], 2500, 20.0, False, 6.0),
    (2, 2, 16, 2, 64, [20000, 16500], 0, 30.0, True, 3.0),    # the split form, row tiles side by side
    (3, 4, 8, 2, 64, [30000, 12345, 5], 11000, 0.0, True, 1.0),
    (1, 1, 16, 2, 64, [40000], 1 << 27, 30.0, False, 3.0),    # a window longer than the cache
])
def test_scored_attention(bits, B, T, G, Hkv, page, lengths, window, cap, slopes, scale):
    g = gen(B * 100 + T + page)
    cache = make_cache(g, B, max(max(lengths), 1) + 20, Hkv, page, bits, k_exp=1 if bits == 4 else 0, v_exp=-1 if bits == 4 else 0)
    Hq = G * Hkv
    q = (normal(g, B, T, Hq, 64) * scale)
    s = slopes_of(Hq) if slopes else None
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((B, T, Hq, 64), 7.0, dtype=dtype, device=DEV)
        ws = pisa.cache_workspace(cache)
        got = pisa.cache_attention(q, cache, i32(lengths), out=out, workspace=ws, cap=cap, slopes=s, window=window)
        assert status(ws) == 0
        check(got, expected(q, cache, lengths, window, cap, s, dtype))


@pytest.mark.parametrize("bits", [16, 4])
def test_scores_with_listed_blocks(bits):
    """A selection's blocks that lie before the window, or cross its border."""
    g = gen(3)
    cache = make_cache(g, 2, 1100, 2, 64, bits)
    q, lengths = normal(g, 2, 1, 16, 64) * 2, [1090, 200]
    idx = i32([[[0, 4, 9, 16, 17], [16, 3, -1, 2, 15]], [[3, 0, -1, -1, -1], [1, 2, 3, -1, -1]]])
    check_listed(cache, q, lengths, idx, 150, 4.0, slopes_of(16))
    # far blocks alone: the bias of the nearest one would drown the scores in 32 bits
    cache = make_cache(g, 2, 90000, 2, 64, bits)
    idx = i32([[[0, 4, 9, -1], [2, 1, -1, 700]], [[3, 0, -1, -1], [1, 2, 3, 1200]]])
    check_listed(cache, q, [90000, 77000], idx, 0, 0.0, slopes_of(16) * 4)
    check_listed(cache, q, [90000, 77000], idx, 0, 3.0, slopes_of(16))


def check_listed(cache, q, lengths, idx, window, cap, s):
    bits = cache.bits
    ws = pisa.cache_workspace(cache)
    got = pisa.cache_attention(q, cache, i32(lengths), idx=idx, workspace=ws, cap=cap, slopes=s, window=window)
    assert status(ws) == 0
    for b in range(2):
        n = lengths[b]
        k, v = ref.tokens(cache, b, n)
        for kv in range(2):
            listed = torch.zeros(n, dtype=torch.bool, device=DEV)
            for x in idx[b, kv].tolist():
                if x >= 0:
                    listed[64 * x:64 * x + 64] = True
            if window:
                listed[:max(0, n - window)] = False
            at = listed.nonzero()[:, 0]
            heads = slice(8 * kv, 8 * kv + 8)
            if at.numel() == 0:
                assert not got[b, 0, heads].any()
                continue
            x = q[b, 0, heads].double() @ k[at, kv].T / 8
            x = (cap * torch.tanh(x / cap) if cap else x) - s[heads, None].double() * (n - 1 - at)
            p = torch.softmax(x, -1)
            o, pv = p @ v[at, kv], p @ v[at, kv].abs()
            big = (q[b, 0, heads].double().abs() @ k[at, kv].abs().T / 8).amax(1, keepdim=True)
            tol = score_ref.tolerance(o, pv, big, n, 2.0 ** (-16 if bits == 16 else -11), torch.bfloat16, cap)
            tol = tol + 2.0 ** -35 * v[at, kv].abs().sum(0)
            assert bool(((got[b, 0, heads].double() - o).abs() <= tol).all())


@pytest.mark.parametrize("T", [1, 5])
def test_tokens_before_the_window_do_not_matter(T):
    """Infinities and NaNs before the window and between the queries' windows, and pages that were given away."""
    g = gen(T)
    lengths, window = [400, 90], 70
    cache = make_cache(g, 2, 420, 2, 16, 16)
    q = normal(g, 2, T, 8, 64)
    n = i32(lengths)
    clean = pisa.cache_attention(q, cache, n, window=window).clone()
    for b, L in enumerate(lengths):
        for p in list(range(0, L - T + 1 - window)) + list(range(L, 420)):  # seen by no query
            page, u = int(cache.table[b, p // 16]), p % 16
            cache.pages[page, :, 0, :, u] = INF if p % 2 else NAN
        for e in range((L - T + 1 - window) // 16):
            cache.table[b, e] = -5 if e % 2 else 1 << 30
    ws = pisa.cache_workspace(cache)
    got = pisa.cache_attention(q, cache, n, window=window, workspace=ws)
    assert status(ws) == 0 and torch.equal(got, clean)
    # the first token of the first query's window is seen by that query alone
    if T > 1:
        p = lengths[0] - T + 1 - window
        cache.pages[int(cache.table[0, p // 16]), :, 0, 1, p % 16] = INF
        got = pisa.cache_attention(q, cache, n, window=window)
        assert bool(torch.isinf(got[0, 0]).all()) and torch.equal(got[0, 1:], clean[0, 1:])
        cache.table[0, p // 16] = -1  # a page that holds it: NaN for those that see a token of it
        got = pisa.cache_attention(q, cache, n, window=window, workspace=ws)
        sees = [t for t in range(T) if lengths[0] - T + t - window + 1 < (p // 16 + 1) * 16]
        for t in range(T):
            assert bool(torch.isnan(got[0, t]).all()) == (t in sees)
        assert status(ws) == 6


def test_capped_infinities():
    """An infinite product counts as plus or minus the cap; without one the row is NaN."""
    g = gen(9)
    cache = make_cache(g, 1, 64, 1, 64, 16)
    cache.pages[:, :, :, 0] = 1.0
    page = int(cache.table[0, 0])
    cache.pages[page, 0, 0, 0, 3] = INF
    cache.pages[page, 0, 0, 0, 9] = -INF
    q = torch.full((1, 1, 1, 64), 0.25, dtype=torch.bfloat16, device=DEV)
    n, cap = i32([20]), 3.0
    got = pisa.cache_attention(q, cache, n, cap=cap, out=torch.empty(1, 1, 1, 64, device=DEV))
    x = torch.full((20,), 2.0, dtype=torch.float64, device=DEV)
    x = cap * torch.tanh(x / cap)
    x[3], x[9] = cap, -cap
    v = cache.pages[page, 0, 0, 1, :20].double()
    o = torch.softmax(x, 0) @ v
    assert bool(((got[0, 0, 0].double() - o).abs() <= 1e-5 * (torch.softmax(x, 0) @ v.abs())).all())
    assert bool(torch.isnan(pisa.cache_attention(q, cache, n, window=30)).all())


@pytest.mark.parametrize("cap", [2.0 ** -20, 5.0, 500.0, 2.0 ** 20])
@pytest.mark.parametrize("slopes", [False, True])
def test_huge_queries_and_keys_of_zero(cap, slopes):
    """4-bit keys of zero have scores of zero whatever the queries are, the others plus or minus the cap."""
    g = gen(31)
    cache = make_cache(g, 1, 256, 1, 64, 4, k_exp=10)
    n, T = 200, 3
    cache.pages.view(cache.pages.shape[0], 144, 32)[:, 0:64:3] = 0  # codes of keys: every third is zero
    k, v = ref.tokens(cache, 0, n)
    q = torch.sign(normal(g, 1, T, 4, 64)) * 2.0 ** 124
    q[:, 1] = 0.0
    q[:, 2, :, 1:] = 0.0
    q = q.to(torch.bfloat16)
    s = slopes_of(4) if slopes else None
    at = n - T + torch.arange(T, device=DEV)
    o, pv, big = score_ref.attention(q[0].double(), k, v, at, torch.zeros_like(at), at + 1, cap, s)
    # products are zero or past the cap; weights of 2^-11, of all tokens (the sum and the weights), and the result's step
    tol = 2 * (2.0 ** -11 + 2.0 ** -16 + 32 * 2.0 ** -24 * cap) * pv + 2.0 ** -8 * (o.abs() + pv * 2.0 ** -9)
    tol += 2.0 ** -25 * v.abs().sum(0)  # fp16 weights' steps
    prompt = pisa.cache_prompt_attention(q, cache, i32([n - T]), cap=cap, slopes=s)
    token = pisa.cache_attention(q, cache, i32([n]), cap=cap, slopes=s)
    for got in (prompt, token):
        assert bool(((got[0].double() - o).abs() <= tol).all()), float(((got[0].double() - o).abs() / tol).max())


def test_zero_scores_are_plain_attention():
    """No cap, no slopes and no window is the plain call, to the bit; a window that holds everything is close."""
    g = gen(4)
    cache = make_cache(g, 2, 3000, 2, 64, 4)
    q, n = normal(g, 2, 2, 32, 64), i32([3000, 77])
    plain = pisa.cache_attention(q, cache, n)
    assert torch.equal(plain, pisa.cache_attention(q, cache, n, cap=0.0, slopes=None, window=0))
    near = pisa.cache_attention(q, cache, n, window=3000)
    assert bool(((near - plain).abs() <= 2.0 ** -7 * plain.abs().amax()).all())


def test_refusals():
    g = gen(5)
    cache = make_cache(g, 2, 40, 2, 16, 16)
    q, n = normal(g, 2, 1, 8, 64), i32([30, 20])
    for kw in (dict(slopes=torch.zeros(7, device=DEV)), dict(slopes=torch.zeros(8)), dict(window=-1),
               dict(slopes=torch.zeros(8, dtype=torch.float64, device=DEV))):
        with pytest.raises(ValueError):
            pisa.cache_attention(q, cache, n, **kw)
    for cap in (-1.0, NAN, INF, 1e-30, 1e30):
        with pytest.raises(pisa.PisaError):
            pisa.cache_attention(q, cache, n, cap=cap)
