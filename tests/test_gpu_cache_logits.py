"""Attention over the cache where logits are large, and query rows whose elements are."""
import pytest
import torch

import cache_ref as ref
import pyramid_top_block_gb300 as pisa
import test_gpu_cache as base

pytestmark = pytest.mark.gpu
DEV = base.DEV


def check_one_hot(cache, q, n, out, idx_blocks=None):
    """Rows whose largest logit is so far above the others that one key has all the weight: its value.

    A logit is off by at most 128 * 2^-24 of the sum of its products' sizes (`big`), so where the two largest
    differ by more than 2^-15 big + 64, every other weight is below e^-64.  The one key's weight is rounded for the
    product with V (2^-11 in fp16, 2^-16 in two bf16 parts) and the result once; the other n keys add e^-64 < 2^-92
    of their values at the most."""
    k, v = ref.tokens(cache, 0, n)
    seen = torch.ones(n, dtype=torch.bool, device=DEV)
    if idx_blocks is not None:
        seen[:] = False
        for b in idx_blocks:
            seen[64 * b:64 * b + 64] = True
    G = q.shape[2] // cache.Hkv
    checked = 0
    for r in range(q.shape[2]):
        kk, vv = k[seen, r // G], v[seen, r // G]
        z = (kk * q[0, 0, r].double()).sum(-1) / 8
        big = float((kk * q[0, 0, r].double()).abs().sum(-1).max() / 8)
        top = z.topk(min(2, z.numel())).values
        o = out[0, 0, r].double()
        assert bool(torch.isfinite(o).all()), r
        if top.numel() == 2 and float(top[0] - top[1]) < 2.0 ** -15 * big + 64:
            continue
        want = vv[int(z.argmax())]
        tol = want.abs() * (2.0 ** -11 if cache.bits == 4 else 2.0 ** -16) + n * 2.0 ** -92 * vv.abs().max()
        tol = tol + torch.finfo(out.dtype).eps / 2 * (want.abs() + tol)
        assert bool(((o - want).abs() <= tol).all()), r
        checked += 1
    assert checked >= q.shape[2] * 3 // 4, checked


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("n", [1, 200, 9000])
def test_large_logits(bits, n):
    """Logits of 2^22 to 2^117: 32 bits hold them, and their differences decide."""
    g = base.gen(n + bits)
    cache = base.make_cache(g, 1, max(n, 640), 2, 64, bits)
    wide = base.in_a_wide_table(cache)
    for e in (22, 25, 27, 30, 33, 36, 40, 64, 96, 112):
        q = base.normal(g, 1, 1, 32, 64) * 2.0 ** e
        for c in (cache, wide):
            for dtype in (torch.bfloat16, torch.float32):
                out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
                pisa.cache_attention(q, c, base.i32([n]), out=out)
                check_one_hot(cache, q, n, out)
        blocks = list(range(min(10, -(-n // 64))))
        idx = base.i32(blocks[::-1]).expand(1, 2, 1, len(blocks)).contiguous()
        check_one_hot(cache, q, n, pisa.cache_attention(q, cache, base.i32([n]), idx=idx), blocks)


@pytest.mark.parametrize("bits", [16, 4])
def test_large_logits_beside_ordinary_rows(bits):
    """A row of large logits in a tile, one of large negative ones, and ordinary rows, which are as ever."""
    g = base.gen(31)
    n, big = 5000, 2.0 ** 40
    cache = base.make_cache(g, 1, n, 1, 64, bits)
    q = base.normal(g, 1, 1, 16, 64)
    mixed = q.clone()
    mixed[0, 0, 3] *= big
    mixed[0, 0, 11] *= -big
    out = pisa.cache_attention(mixed, cache, base.i32([n]))
    for r in range(16):
        if r not in (3, 11):
            base.check_attention(cache, q[:, :, r:r + 1], [n], out[:, :, r:r + 1])
    assert bool(torch.isfinite(out).all())
    # all logits large, of one sign, and equal: the mean of the values
    k = torch.full((1, n, 1, 64), -1.5, dtype=torch.bfloat16, device=DEV)
    v = base.normal(g, 1, n, 1, 64)
    pisa.cache_append(None, k, v, cache, base.i32([0]), None)
    _, vv = ref.tokens(cache, 0, n)
    mean, size = vv[:, 0].mean(0), vv[:, 0].abs().mean(0)
    for sign in (1.0, -1.0):
        q = torch.full((1, 1, 16, 64), sign * 2.0 ** 100, dtype=torch.bfloat16, device=DEV)
        out = pisa.cache_attention(q, cache, base.i32([n]))[0, 0].double()
        # equal weights, rounded alike; fp32 sums of n terms
        tol = n * 2.0 ** -23 * size + 2.0 ** -11 * size + 2.0 ** -9 * mean.abs()
        assert bool(((out - mean).abs() <= tol).all())


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("e", [100, 114, 116, 120, 125])
def test_query_rows_up_to_the_end_of_the_range(bits, e):
    """Elements up to 2^127 over keys that are small enough for the logits to fit 32 bits."""
    g = base.gen(e + bits)
    n = 300
    cache = base.make_cache(g, 1, n, 2, 64, bits, k_exp=-24 if bits == 4 else 0)
    if bits == 16:
        cache.pages[:, :, :, 0] *= 2.0 ** -24
    q = (base.normal(g, 1, 1, 32, 64).clamp(-3.9, 3.9) * 2.0 ** e)
    assert bool(torch.isfinite(q).all())
    for c in (cache, base.in_a_wide_table(cache)):
        check_one_hot(cache, q, n, pisa.cache_attention(q, c, base.i32([n])))
    blocks = [4, 0, 3]
    idx = base.i32(blocks).expand(1, 2, 1, 3).contiguous()
    check_one_hot(cache, q, n, pisa.cache_attention(q, cache, base.i32([n]), idx=idx), blocks)


@pytest.mark.parametrize("bits", [16, 4])
def test_large_queries_over_keys_of_zero(bits):
    """Logits of zero stay zero, whatever the exponents: the mean of the values."""
    g = base.gen(33)
    n = 200
    for k_exp in ((0, 24) if bits == 4 else (0,)):
        cache = base.make_cache(g, 1, n, 1, 64, bits, k_exp=k_exp)
        v = base.normal(g, 1, n, 1, 64)
        pisa.cache_append(None, torch.zeros_like(v), v, cache, base.i32([0]), None)
        _, vv = ref.tokens(cache, 0, n)
        mean, size = vv[:, 0].mean(0), vv[:, 0].abs().mean(0)
        q = base.normal(g, 1, 1, 16, 64).clamp(-3.9, 3.9) * 2.0 ** 125
        out = pisa.cache_attention(q, cache, base.i32([n]))[0, 0].double()
        tol = n * 2.0 ** -23 * size + 2.0 ** -11 * size + 2.0 ** -9 * mean.abs()
        assert bool(((out - mean).abs() <= tol).all()), k_exp


@pytest.mark.parametrize("bits", [16, 4])
def test_an_infinite_element_beside_large_ones(bits):
    """Every logit is minus infinity, whatever the row's finite elements are: zeros."""
    g = base.gen(34)
    n = 200
    cache = base.make_cache(g, 1, n, 1, 64, bits)
    k = base.normal(g, 1, n, 1, 64)
    k[..., 7] = -1.0
    pisa.cache_append(None, k, base.normal(g, 1, n, 1, 64), cache, base.i32([0]), None)
    q = base.normal(g, 1, 1, 16, 64) * 2.0 ** 20
    q[..., 7] = float("inf")
    ordinary = base.normal(g, 64)
    q[0, 0, 5] = ordinary
    out = pisa.cache_attention(q, cache, base.i32([n]))
    rows = [r for r in range(16) if r != 5]
    assert bool((out[0, 0, rows] == 0).all())
    base.check_attention(pisa.PagedCache(cache.pages, cache.table, 64), ordinary.expand(1, 1, 1, 64), [n],
                         out[:, :, 5:6])


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("T,G,page,n", [(5, 8, 16, 130), (5, 8, 16, 3), (3, 16, 64, 9001), (16, 4, 32, 2059)])
def test_large_logits_of_several_queries(bits, T, G, page, n):
    """Each query has its own last token, rows that see nothing share the tile, NaNs lie behind all of them."""
    g = base.gen(n + T)
    cache = base.make_cache(g, 1, max(n + 20, 70), 1, page, bits)
    for p in range(n, n + 20):
        base.poison(cache, 0, p)
    for e in (24, 31, 50, 110):
        q = base.normal(g, 1, T, G, 64)
        q[:, :, 1:] *= 2.0 ** e  # the first row of each query stays ordinary
        for c in (cache, base.in_a_wide_table(cache)):
            out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
            pisa.cache_attention(q, c, base.i32([n]), out=out)
            for t in range(T):
                see = n - T + t + 1
                if see <= 0:
                    assert bool((out[0, t] == 0).all())
                else:
                    check_one_hot(cache, q[:, t:t + 1, 1:], see, out[:, t:t + 1, 1:])
            base.check_attention(cache, q[:, :, :1], [n], out[:, :, :1])
