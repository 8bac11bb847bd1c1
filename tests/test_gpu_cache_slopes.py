"""Biases by distance of any size and sign, at far positions too, against 64 bits."""
import pytest
import torch

import cache_ref as ref
import pyramid_top_block_gb300 as pisa
import score_ref
from test_gpu_cache import DEV, gen, i32, make_cache, normal, status

pytestmark = pytest.mark.gpu


def f32(x):
    return torch.tensor(x, dtype=torch.float32, device=DEV)


def expected(q, k, v, at, lo, hi, cap, slopes, weight, dtype):
    """(o, tolerance): score_ref's, its sums over the keys that count, those of at least 2^-40 of the row's largest weight.
    The others are off by at most themselves, so by 2^-40 sum |v| and, of the sum of weights, by n 2^-40 <= 2^-20 for
    n <= 2^20, twice.  fp16 weights (4-bit pages) have steps of 2^-24 at least, relative to a reference of at most the largest
    one, so those that count are also off by 2^-25 each."""
    G = q.shape[1] // k.shape[1]
    o, pv, big = score_ref.attention(q, k, v, at, lo, hi, cap, slopes)
    x = torch.einsum("thd,nhd->thn", q, k.repeat_interleave(G, 1)) / 8
    if cap:
        x = cap * torch.tanh(x / cap)
    j = torch.arange(k.shape[0], device=DEV)
    x = x - slopes.double()[:, None] * (at[:, None, None] - j).abs()
    x = torch.where(((j >= lo[:, None]) & (j < hi[:, None]))[:, None], x, -float("inf"))
    count = (x >= x.amax(-1, keepdim=True) - 40 * 0.6931472).double()
    tol = score_ref.tolerance(o, pv, big, count.sum(-1, keepdim=True), weight, dtype, cap)
    a = v.abs().repeat_interleave(G, 1)
    return o, tol + 2.0 ** -19 * pv + 2.0 ** -40 * a.sum(0) + 2.0 ** -25 * torch.einsum("thn,nhd->thd", count, a)


def check(got, want):
    o, tol = want
    off = (got.double() - o).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (bad.nonzero()[0].tolist(), float((off / tol)[bad].nan_to_num(nan=1e30).max()))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("cap", [0.0, 40.0, 300.0])
@pytest.mark.parametrize("n,T", [(120000, 20), (131072, 3), (2500, 200)])
def test_steep_slopes_over_long_caches(bits, cap, n, T):
    """Short chunks whose key tiles are taken in pieces: a piece of far tokens alone has large negative logits."""
    g = gen(T)
    cache = make_cache(g, 1, n + 5, 1, 64, bits)
    q, s = normal(g, 1, T, 4, 64) * 3, f32([300.0, 1000.0, 3000.0, 10000.0])
    k, v = ref.tokens(cache, 0, n)
    at = n - T + torch.arange(T, device=DEV)
    zero = torch.zeros_like(at)
    got = pisa.cache_prompt_attention(q, cache, i32([n - T]), cap=cap, slopes=s)
    check(got[0], expected(q[0].double(), k, v, at, zero, at + 1, cap, s, 2.0 ** (-8 if bits == 16 else -11), torch.bfloat16))
