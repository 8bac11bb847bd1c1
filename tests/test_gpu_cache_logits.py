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
