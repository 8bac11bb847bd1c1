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
    """(o, tolerance): score_ref's, its sums over the keys that count, those of at least 2^-40 of the row's largest
    weight.  The others are off by at most themselves, so by 2^-40 sum |v| and, of the sum of weights, by n 2^-40 <=
    2^-20 for n <= 2^20, twice.  fp16 weights (4-bit pages) have steps of 2^-24 at least, relative to a reference of at
    most the largest one, so those that count are also off by 2^-25 each.  (Positions as doubles: whole numbers times a
    float are 32 bits.)"""
    G = q.shape[1] // k.shape[1]
    o, pv, big = score_ref.attention(q, k, v, at.double(), lo, hi, cap, slopes)
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


def both(q, cache, n, T, cap, s, window=0):
    """The newest T tokens by the prompts' call and by the single tokens' (bf16 and 32 bits), checked."""
    k, v = ref.tokens(cache, 0, n)
    at = n - T + torch.arange(T, device=DEV)
    lo = (at - window + 1).clamp(min=0) if window else torch.zeros_like(at)
    bf16 = cache.bits == 16
    for dtype, weight in ((torch.bfloat16, 2.0 ** (-16 if bf16 else -11)),
                          (torch.float32, 2.0 ** (-22 if bf16 else -20))):
        out = torch.full((1, T, q.shape[2], 64), 7.0, dtype=dtype, device=DEV)
        got = pisa.cache_attention(q, cache, i32([n]), out=out, cap=cap, slopes=s, window=window)
        check(got[0], expected(q[0].double(), k, v, at, lo, at + 1, cap, s, weight, dtype))
    got = pisa.cache_prompt_attention(q, cache, i32([n - T]), cap=cap, slopes=s, window=window)
    check(got[0], expected(q[0].double(), k, v, at, lo, at + 1, cap, s, 2.0 ** (-8 if bf16 else -11), torch.bfloat16))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("cap", [0.0, 40.0, 300.0])
@pytest.mark.parametrize("n,T,window", [(90000, 3, 0), (1000, 16, 0), (30000, 2, 9000), (50, 5, 20)])
def test_negative_slopes(bits, cap, n, T, window):
    """Biases that grow with the distance: the first tokens in sight count, whose own bias is large."""
    g = gen(n + T)
    cache = make_cache(g, 1, n + 5, 1, 64, bits)
    both(normal(g, 1, T, 8, 64) * 3, cache, n, T, cap, f32([-30.0, -4.0, -1.0, -0.1, 0.1, 1.0, 4.0, 30.0]), window)


@pytest.mark.parametrize("bits", [16, 4])
def test_negative_slopes_of_prefixes(bits):
    """Tokens behind a query in sight, the farthest ones there or before it."""
    g = gen(3)
    T, start = 700, 300
    cache = make_cache(g, 1, start + T, 1, 64, bits)
    q, s = normal(g, 1, T, 4, 64) * 3, f32([-8.0, -0.5, -0.02, 0.5])
    last = torch.maximum(start + torch.arange(T) + 1, torch.tensor(start + 500)).to(torch.int32)[None].to(DEV)
    k, v = ref.tokens(cache, 0, start + T)
    at = start + torch.arange(T, device=DEV)
    for cap in (0.0, 50.0):
        got = pisa.cache_prompt_attention(q, cache, i32([start]), last=last, cap=cap, slopes=s)
        check(got[0], expected(q[0].double(), k, v, at, torch.zeros_like(at), last[0].long(), cap, s,
                               2.0 ** (-8 if bits == 16 else -11), torch.bfloat16))


@pytest.mark.parametrize("bits", [16, 4])
def test_negative_slopes_of_listed_blocks(bits):
    g = gen(4)
    n = 80000
    cache = make_cache(g, 1, n, 1, 64, bits)
    q, s = normal(g, 1, 1, 4, 64) * 3, f32([-10.0, -1.0, -0.05, 1.0])
    blocks = [1000, 500, 777, 1200, 501]
    at = torch.cat([torch.arange(64 * x, 64 * x + 64) for x in blocks]).sort().values.to(DEV)
    k, v = ref.tokens(cache, 0, n)
    keep = torch.zeros(n, dtype=torch.bool, device=DEV)
    for window, cap in ((0, 0.0), (0, 20.0), (n - 64 * 501 - 7, 0.0)):
        keep.zero_()
        keep[at] = True
        if window:
            keep[:n - window] = False
        j = keep.nonzero()[:, 0]
        got = pisa.cache_attention(q, cache, i32([n]), idx=i32([[blocks + [-1]]]), cap=cap, slopes=s, window=window)
        x = q[0, 0].double() @ k[j, 0].T / 8
        x = (cap * torch.tanh(x / cap) if cap else x) - s.double()[:, None] * (n - 1 - j)
        p = torch.softmax(x, -1)
        o, pv = p @ v[j, 0], p @ v[j, 0].abs()
        big = (q[0, 0].double().abs() @ k[j, 0].abs().T / 8).amax(1, keepdim=True)
        tol = score_ref.tolerance(o, pv, big, j.numel(), 2.0 ** (-16 if bits == 16 else -11), torch.bfloat16, cap)
        check(got[0, 0], (o, tol + 2.0 ** -25 * v[j, 0].abs().sum(0)))


@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_negative_slopes_past_two_to_the_24(cap):
    """Distances that 32 bits do not hold exactly, between tokens that count.  All entries of the table hold one of
    a few pages, so that the cache is small."""
    g = gen(5)
    n, T, page, few = (1 << 24) + 5000, 3, 256, 8
    for bits in (16, 4):
        small = make_cache(g, 1, few * page, 1, page, bits)
        e = torch.arange(-(-n // page), device=DEV)
        table = small.table[0, e % few][None].contiguous()
        cache = pisa.PagedCache(small.pages, table, page)
        q, s = normal(g, 1, T, 2, 64) * 6, f32([-0.5, -2.0])
        m = 500  # tokens that can count: the others' bias is 100 less, which the scores (below 40) do not make up for
        k, v = ref.tokens(cache, 0, m)
        at = n - T + torch.arange(T, device=DEV)
        zero = torch.zeros_like(at)
        weight = 2.0 ** (-8 if bits == 16 else -11)
        want = expected(q[0].double(), k, v, at, zero, zero + m, cap, s, weight, torch.bfloat16)
        check(pisa.cache_prompt_attention(q, cache, i32([n - T]), cap=cap, slopes=s)[0], want)
        check(pisa.cache_attention(q, cache, i32([n]), cap=cap, slopes=s)[0], want)


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
    weight = 2.0 ** (-8 if bits == 16 else -11)
    check(got[0], expected(q[0].double(), k, v, at, zero, at + 1, cap, s, weight, torch.bfloat16))


@pytest.mark.parametrize("bits,size", [(16, 1.0), (4, 1.0), (4, 2.0 ** -75)])
@pytest.mark.parametrize("cap", [0.0, 40.0])
def test_slopes_of_any_size(bits, size, cap):
    """The header asks for finite ones alone."""
    g = gen(8)
    n, T = 5000, 4
    cache = make_cache(g, 1, n, 1, 64, bits, k_exp=-24 if size < 1 else 0)
    q = (normal(g, 1, T, 8, 64) * size).to(torch.bfloat16)
    for s in ([1e5, -1e5, 1e12, -1e12, 1e30, -1e30, 3e38, -3e38],
              [1e-30, -1e-30, 1e-44, -1e-44, 0.0, -0.0, 1e-20, -1e-20]):
        both(q, cache, n, T, cap, f32(s))


def test_slopes_of_huge_queries_over_keys_of_zero():
    """4-bit keys of zero have scores of zero whatever the queries are, so that the bias alone decides."""
    g = gen(10)
    n, T = 3000, 3
    cache = make_cache(g, 1, n, 1, 64, 4, k_exp=10)
    cache.pages.view(cache.pages.shape[0], 144, 32)[:, 0:64] = 0
    q = (torch.sign(normal(g, 1, T, 4, 64)) * 2.0 ** 126).to(torch.bfloat16)
    both(q, cache, n, T, 0.0, f32([0.002, -0.003, 0.7, 1e-5]))


def test_positions_past_the_table_with_slopes():
    """Starts at both ends of 32 bits: flagged, and what is in sight still counts by the tokens' distances."""
    g = gen(9)
    for bits in (16, 4):
        cache = make_cache(g, 1, 512, 1, 64, bits)
        n, T = 512, 12
        q, s = normal(g, 1, T, 4, 64) * 3, f32([0.05, -0.05, 1.0, 0.0])
        k, v = ref.tokens(cache, 0, n)
        for cap in (0.0, 6.0):
            for start, last in (((1 << 31) - 16, None), (-(1 << 31) + 8, [[0, 5, 512] * 4])):
                at = start + torch.arange(T, device=DEV)
                hi = torch.full_like(at, n)
                ws = pisa.cache_workspace(cache)
                got = pisa.cache_prompt_attention(q, cache, i32([start]), last=None if last is None else i32(last),
                                                  cap=cap, slopes=s, workspace=ws)
                assert status(ws) == 6
                if last is not None:  # (no token of the sequence is there: it ends before 0)
                    assert not bool(got.any())
                    continue
                check(got[0], expected(q[0].double(), k, v, at, torch.zeros_like(at), hi, cap, s,
                                       2.0 ** (-8 if bits == 16 else -11), torch.bfloat16))
