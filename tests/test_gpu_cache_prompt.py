"""Attention of a prompt's tokens over the paged cache, against 64 bits."""
import pytest
import torch

import cache_ref as ref
import pyramid_top_block_gb300 as pisa
import score_ref
from test_gpu_cache import DEV, gen, i32, make_cache, normal, status
from test_gpu_cache_scores import slopes_of

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def expected(q, cache, start, counts, first=None, last=None, window=0, cap=0.0, slopes=None):
    B, T, Hq, _ = q.shape
    o = torch.full((B, T, Hq, 64), 7.0, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(o)
    for b in range(B):
        m, n = counts[b], start[b] + counts[b]
        if m == 0:
            continue
        k, v = ref.tokens(cache, b, n)
        at = start[b] + torch.arange(m, device=DEV)
        lo = torch.zeros_like(at) if first is None else first[b, :m].long()
        hi = at + 1 if last is None else last[b, :m].long().clamp(max=n)
        if window:
            lo = torch.maximum(lo, at - window + 1)
        x, pv, big = score_ref.attention(q[b, :m].double(), k, v, at, lo, hi, cap, slopes)
        o[b, :m] = x
        tol[b, :m] = score_ref.tolerance(x, pv, big, n, 2.0 ** (-8 if cache.bits == 16 else -11), torch.bfloat16, cap)
        if cache.bits == 4:  # fp16 weights' steps (see ref.tolerance)
            tol[b, :m] += 2.0 ** -25 * v.abs().sum(0).repeat_interleave(Hq // cache.Hkv, 0)
    return o, tol


def check(got, want):
    o, tol = want
    off = (got.double() - o).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (bad.nonzero()[0].tolist(), float((off / tol.clamp(min=1e-30))[bad].max()))


def spans(kind, start, counts, T, seed=0):
    """(first, last) int32 [B, T] or None; rows behind a count hold nonsense."""
    B = len(start)
    g = torch.Generator().manual_seed(seed)
    if kind == "causal":
        return None, None
    at = torch.tensor(start)[:, None] + torch.arange(T)
    first = torch.full((B, T), -3, dtype=torch.int32)
    last = (at + 1).to(torch.int32)
    if kind == "documents":
        for b in range(B):
            begin = 0
            for t in range(counts[b]):
                if t and float(torch.rand(1, generator=g)) < 0.03:
                    begin = start[b] + t
                first[b, t] = begin
        last = None
    elif kind == "prefix":
        edge = torch.tensor(start) + (torch.tensor(counts) + 1) // 2
        last = torch.maximum(at + 1, edge[:, None]).to(torch.int32)
        first = None
    else:  # anything, empty ones and ones past the ends among them
        n = int(max(a + c for a, c in zip(start, counts)))
        first = torch.randint(-5, n + 5, (B, T), generator=g, dtype=torch.int32)
        last = first + torch.randint(-40, n, (B, T), generator=g, dtype=torch.int32)
    for x in (first, last):
        if x is not None:
            for b in range(B):
                x[b, counts[b]:] = 1 << 30
    return tuple(None if x is None else x.to(DEV).contiguous() for x in (first, last))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("B,T,G,Hkv,page,start,counts,kind,window,cap,slopes", [
    (1, 1, 1, 1, 16, [0], [1], "causal", 0, 0.0, False),
    (1, 1, 16, 2, 64, [700], [1], "causal", 0, 0.0, False),
    (2, 33, 4, 2, 64, [0, 5], [33, 20], "causal", 0, 0.0, False),
    (1, 300, 16, 2, 64, [0], [300], "causal", 0, 0.0, False),
    (1, 129, 8, 1, 32, [1000], [129], "causal", 0, 30.0, False),
    (2, 257, 2, 3, 128, [77, 3], [257, 0], "causal", 0, 0.0, True),
    (1, 640, 4, 1, 64, [0], [640], "documents", 0, 0.0, False),
    (2, 200, 16, 1, 16, [10, 400], [200, 111], "prefix", 0, 20.0, True),
    (1, 500, 1, 2, 256, [300], [500], "causal", 37, 0.0, False),
    (1, 130, 8, 2, 64, [4000], [130], "causal", 1000, 5.0, True),
    (3, 65, 4, 2, 32, [0, 200, 31], [65, 64, 1], "any", 0, 0.0, False),
    (2, 190, 16, 2, 64, [3, 900], [190, 150], "any", 50, 10.0, True),
    (1, 17, 16, 1, 64, [30000], [17], "causal", 0, 0.0, False),
    (1, 1100, 16, 1, 64, [1500], [1100], "causal", 0, 0.0, False),
    (2, 300, 4, 2, 64, [700, 0], [300, 280], "prefix", 0, 0.0, True),
    (1, 400, 2, 1, 128, [100], [400], "any", 0, 0.0, True),
    (1, 700, 8, 1, 64, [0], [700], "documents", 200, 0.0, True),
    (1, 300, 16, 1, 64, [200], [300], "causal", 0, 2.0, False),      # scores past the cap
    (1, 200, 4, 1, 64, [100], [200], "prefix", 0, 300.0, False),
    (1, 200, 4, 1, 64, [100], [200], "causal", 0, 0.75, True),
    (2, 530, 16, 1, 64, [6000, 12000], [530, 100], "causal", 0, 8.0, True),
    (1, 40, 16, 1, 64, [20000], [40], "prefix", 0, 0.0, False),      # listed spans, in pieces
    (2, 20, 8, 2, 128, [9000, 17000], [20, 9], "any", 0, 0.0, True),
    (1, 90, 4, 1, 16, [12345], [90], "documents", 7000, 30.0, False),
    (2, 18, 16, 3, 32, [25000, 300], [18, 18], "causal", 0, 0.0, False),
    (40, 3, 4, 2, 64, [11 * b for b in range(40)], [b % 4 for b in range(40)], "causal", 0, 0.0, False),
])
def test_prompt_attention(bits, B, T, G, Hkv, page, start, counts, kind, window, cap, slopes):
    g = gen(T * 10 + page)
    cap_tokens = max(a + T for a in start) + 3
    cache = make_cache(g, B, cap_tokens, Hkv, page, bits, k_exp=-1 if bits == 4 else 0, v_exp=1 if bits == 4 else 0, layers=2)
    Hq = G * Hkv
    # queries inside a fused projection's rows
    q = (normal(g, B, T, Hq + 2 * Hkv, 64) * (3.0 if cap else 1.0))[:, :, :Hq]
    s = slopes_of(Hq) if slopes else None
    first, last = spans(kind, start, counts, T, seed=T)
    out = torch.full((B, T, Hq, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = pisa.cache_workspace(cache)
    got = pisa.cache_prompt_attention(q, cache, i32(start), counts=i32(counts), out=out, workspace=ws, cap=cap, slopes=s,
                                      window=window, first=first, last=last)
    assert got is out and status(ws) == 0
    check(got, expected(q, cache, start, counts, first, last, window, cap, s))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("cap", [20.0, 128.0, 129.0, 40000.0])
def test_scores_below_and_past_a_cap(bits, slopes, cap):
    """Rows whose scores stay far below the cap, come near it and pass it, side by side and far apart."""
    g = gen(int(cap))
    start, T, Hkv, G = 200, 300, 1, 4
    cache = make_cache(g, 1, start + T, Hkv, 64, bits)
    s = slopes_of(G) if slopes else None
    k, _ = ref.tokens(cache, 0, start + T)
    size = float((normal(g, 64, 64).double() @ k[:, 0].T / 8).abs().amax())  # of the largest of many scores
    for scale in (torch.tensor([0.1, 0.4, 0.9, 3.0], device=DEV)[None, :, None].expand(T, G, 1),
                  torch.tensor([0.1, 0.4, 0.9, 3.0], device=DEV)[torch.arange(T, device=DEV) * 4 // T][:, None, None]):
        q = (normal(g, 1, T, G, 64) * (scale * cap / size)).to(torch.bfloat16)
        ws = pisa.cache_workspace(cache)
        got = pisa.cache_prompt_attention(q, cache, i32([start]), workspace=ws, cap=cap, slopes=s)
        assert status(ws) == 0
        check(got, expected(q, cache, [start], [T], cap=cap, slopes=s))


def test_a_prompt_equals_its_tokens_one_by_one():
    """The last sixteen tokens of a prompt, as cache_attention gives them, with the same scores."""
    g = gen(2)
    for bits in (16, 4):
        cache = make_cache(g, 2, 400, 2, 64, bits)
        q, start, s = normal(g, 2, 90, 16, 64) * 2, i32([300, 0]), slopes_of(16)
        a = pisa.cache_prompt_attention(q, cache, start, cap=9.0, slopes=s, window=60)
        b = pisa.cache_attention(q[:, -16:], cache, start + 90, cap=9.0, slopes=s, window=60)
        assert bool(((a[:, -16:].float() - b.float()).abs() <= 2.0 ** -6 * b.float().abs().amax()).all())


@pytest.mark.parametrize("T,G", [(40, 16), (700, 2)])
def test_what_a_query_does_not_see_does_not_matter(T, G):
    """Infinities and NaNs in later tokens, other documents and behind the sequence reach nobody who does not see them."""
    g = gen(T)
    Hkv, start = 2, 37
    n = start + T
    cache = make_cache(g, 1, n + 70, Hkv, 16, 16)
    q = normal(g, 1, T, G * Hkv, 64)
    first, last = spans("documents", [start], [T], T, seed=1)
    clean = pisa.cache_prompt_attention(q, cache, i32([start]), first=first).clone()

    def spoil(p, value, what):
        cache.pages[int(cache.table[0, p // 16]), :, 0, what, p % 16] = value

    for p in range(n, n + 70):
        spoil(p, NAN if p % 2 else INF, 0)
        spoil(p, INF if p % 3 else NAN, 1)
    assert torch.equal(clean, pisa.cache_prompt_attention(q, cache, i32([start]), first=first))
    # a value, then a key, in the middle: its own document's later tokens see it, nobody else does
    p = start + T // 2
    sees = ((first[0] <= p) & (start + torch.arange(T, device=DEV) >= p))
    assert bool(sees.any()) and not bool(sees.all())
    keep = cache.pages.clone()
    for what, value in ((1, INF), (1, -INF), (1, NAN), (0, NAN)):
        cache.pages.copy_(keep)
        spoil(p, value, what)
        got = pisa.cache_prompt_attention(q, cache, i32([start]), first=first)
        assert torch.equal(got[0, ~sees], clean[0, ~sees])
        assert not bool(torch.isfinite(got[0, sees]).any())
    # one dim of one value
    cache.pages.copy_(keep)
    cache.pages[int(cache.table[0, p // 16]), 1, 0, 1, p % 16, 5] = -INF
    got = pisa.cache_prompt_attention(q, cache, i32([start]), first=first)
    want = clean.clone()
    want[0, sees, G:, 5] = -INF
    assert torch.equal(torch.isinf(got), torch.isinf(want)) and bool((got[torch.isinf(got)] < 0).all())
    fine = ~torch.isinf(want)
    assert torch.equal(got[fine], want[fine])


def test_pages_out_of_range():
    """A page out of range: NaN for the queries that see a token of it, the others as before; flagged where seen."""
    g = gen(8)
    for bits in (16, 4):
        cache = make_cache(g, 1, 512, 2, 32, bits)
        q, T = normal(g, 1, 300, 8, 64), 300
        ws = pisa.cache_workspace(cache)
        clean = pisa.cache_prompt_attention(q, cache, i32([100]), workspace=ws, window=64).clone()
        cache.table[0, 13:] = -1  # behind the sequence
        assert torch.equal(clean, pisa.cache_prompt_attention(q, cache, i32([100]), workspace=ws, window=64))
        assert status(ws) == 0
        cache.table[0, 6] = 1 << 29  # tokens 192 .. 223
        got = pisa.cache_prompt_attention(q, cache, i32([100]), workspace=ws, window=64)
        at = 100 + torch.arange(T, device=DEV)
        sees = (at >= 192) & (at - 63 <= 223)
        assert bool(torch.isnan(got[0, sees]).all()) and torch.equal(got[0, ~sees], clean[0, ~sees])
        assert status(ws) == 6


def test_rows_that_see_nothing_and_logits_of_minus_infinity():
    g = gen(11)
    cache = make_cache(g, 1, 200, 1, 64, 16)
    q, T = normal(g, 1, 150, 4, 64), 150
    at = torch.arange(T, device=DEV, dtype=torch.int32)[None]
    first = torch.where(at % 3 == 0, at + 1, 0).to(torch.int32).contiguous()  # every third query sees nothing
    got = pisa.cache_prompt_attention(q, cache, i32([0]), first=first)
    assert not bool(got[0, ::3].any()) and bool(torch.isfinite(got).all())
    # all products minus infinity: zeros, as for the single tokens' call
    cache.pages[:, :, :, 0] = -INF
    ones = torch.ones_like(q)
    assert not bool(pisa.cache_prompt_attention(ones, cache, i32([0])).any())
    # one of plus infinity: NaN for those that see it
    cache.pages[:, :, :, 0] = 1.0
    cache.pages[int(cache.table[0, 1]), 0, 0, 0, 6] = INF
    got = pisa.cache_prompt_attention(ones, cache, i32([0]))
    assert bool(torch.isnan(got[0, 70:]).all()) and bool(torch.isfinite(got[0, :70]).all())


def test_large_scores():
    """Scores of thousands to 2^100: one token takes all the weight, whatever the others hold."""
    g = gen(12)
    for bits, scale in ((16, 2.0 ** 40), (4, 2.0 ** 60), (16, 2.0 ** 10), (4, 2.0 ** 12)):
        cache = make_cache(g, 1, 260, 2, 64, bits)
        q = normal(g, 1, 250, 8, 64) * scale
        got = pisa.cache_prompt_attention(q, cache, i32([0]))
        assert bool(torch.isfinite(got).all())
        k, v = ref.tokens(cache, 0, 250)
        x = torch.einsum("thd,nhd->thn", q[0].double(), k.repeat_interleave(4, 1)) / 8
        x = torch.where((torch.arange(250, device=DEV) <= torch.arange(250, device=DEV)[:, None])[:, None], x, -INF)
        two = x.topk(2, -1)
        # clear of the rounding of a sum of 64 products, the largest weight is 1
        mag = torch.einsum("thd,nhd->thn", q[0].double().abs(), k.abs().repeat_interleave(4, 1)).amax(-1) / 8
        sure = two.values[..., 0] - two.values[..., 1] > 100 + 2.0 ** -14 * mag
        assert bool(sure.any())
        want = v.repeat_interleave(4, 1).permute(1, 0, 2)[torch.arange(8, device=DEV), two.indices[..., 0]]
        off = (got[0].double() - want).abs()
        assert bool((off[sure] <= 2.0 ** -7 * want[sure].abs()).all())


def test_large_scores_with_slopes():
    """The same with a bias by distance, which they drown."""
    g = gen(32)
    for bits, scale in ((16, 2.0 ** 30), (4, 2.0 ** 40), (16, 2.0 ** 14), (4, 2.0 ** 16)):
        cache = make_cache(g, 1, 700, 1, 64, bits)
        T, at = 250, 400
        q = normal(g, 1, T, 4, 64) * scale
        s = slopes_of(4)
        for got in (pisa.cache_prompt_attention(q, cache, i32([at]), slopes=s)[0],
                    torch.cat([pisa.cache_attention(q[:, t:t + 10], cache, i32([at + t + 10]), slopes=s)[0]
                               for t in range(0, T, 10)])):
            assert bool(torch.isfinite(got).all())
            k, v = ref.tokens(cache, 0, at + T)
            j, p = torch.arange(at + T, device=DEV), at + torch.arange(T, device=DEV)
            x = torch.einsum("thd,nd->thn", q[0].double(), k[:, 0]) / 8 - s.double()[:, None] * (p[:, None, None] - j).abs()
            x = torch.where((j <= p[:, None])[:, None], x, -INF)
            two = x.topk(2, -1)
            mag = torch.einsum("thd,nd->thn", q[0].double().abs(), k[:, 0].abs()).amax(-1) / 8
            sure = two.values[..., 0] - two.values[..., 1] > 100 + 2.0 ** -14 * mag
            assert bool(sure.any())
            want = v[:, 0][two.indices[..., 0]]
            assert bool(((got.double() - want).abs()[sure] <= 2.0 ** -7 * want[sure].abs()).all())


def test_nobody_sees_anything():
    """Whole row tiles without a token: zeros, whatever the output held; rows behind the count as they were."""
    g = gen(33)
    cache = make_cache(g, 2, 9000, 2, 64, 16)
    for T, start in ((300, [0, 100]), (20, [8000, 70])):
        q = normal(g, 2, T, 8, 64)
        first = torch.full((2, T), 1 << 29, dtype=torch.int32, device=DEV)
        first[1, T // 2:] = 0
        out = torch.full((2, T, 8, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        counts = [T, T - 3]
        pisa.cache_prompt_attention(q, cache, i32(start), counts=i32(counts), first=first, out=out)
        check(out, expected(q, cache, start, counts, first))
        last = torch.zeros(2, T, dtype=torch.int32, device=DEV)
        out.fill_(7.0)
        pisa.cache_prompt_attention(q, cache, i32(start), counts=i32([0, 1]), last=last, out=out)
        assert not bool(out[1, 0].any()) and bool((out[0] == 7).all()) and bool((out[1, 1:] == 7).all())


@pytest.mark.parametrize("T,cap", [(300, 1000), (24, 40000)])
def test_captured_with_other_starts_and_counts(T, cap):
    """A call in a graph, replayed with other contents: both forms of the kernel; two graphs that share a workspace, one
    after the other."""
    g = gen(T)
    for bits in (16, 4):
        cache = make_cache(g, 2, cap, 2, 64, bits)
        q, start, counts = normal(g, 2, T, 8, 64), i32([5, 0]), i32([T, T])
        out, ws = torch.zeros_like(q), pisa.cache_workspace(cache)
        step = lambda: pisa.cache_prompt_attention(q, cache, start, counts=counts, out=out, workspace=ws)  # noqa: E731
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
        for cg in graphs:
            with torch.cuda.graph(cg):
                step()
        for i, (a, c) in enumerate((([cap - T, 3], [T, 2]), ([0, cap // 2], [1, T]), ([cap // 3, 0], [T - 1, 0]))):
            start.copy_(i32(a))
            counts.copy_(i32(c))
            q.copy_(normal(g, 2, T, 8, 64))
            out.fill_(7.0)
            graphs[i % 2].replay()
            check(out, expected(q, cache, a, c))
        assert status(ws) == 0


def test_two_streams_with_workspaces_of_their_own():
    g = gen(41)
    cache = make_cache(g, 1, 30000, 2, 64, 4)
    qs = [normal(g, 1, 40, 16, 64), normal(g, 1, 700, 16, 64)]
    starts = [i32([29000]), i32([100])]
    want = [pisa.cache_prompt_attention(q, cache, s).clone() for q, s in zip(qs, starts)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    wss = [pisa.cache_workspace(cache) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [pisa.cache_prompt_attention(q, cache, s, workspace=w, stream=st)
               for q, s, w, st in zip(qs, starts, wss, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_pages_past_four_gigabytes():
    """Pages of a pool of layers whose distance from the first is more than 2^32 bytes."""
    g = gen(42)
    for bits in (16, 4):
        Hkv, page, n = 2, 256, 1300
        inner = (Hkv, 4, 2, 64, 64) if bits == 16 else (Hkv, 4, 72 * 64)
        per = torch.Size(inner).numel() * (2 if bits == 16 else 1)
        layers = -(-(5 << 30) // (per * 40))  # forty pages of so many layers are more than 5 GB
        pool = torch.empty((40, layers) + inner, dtype=torch.bfloat16 if bits == 16 else torch.uint8, device=DEV)
        small = make_cache(g, 1, n, Hkv, page, bits)
        table = torch.arange(39, 39 - small.table.shape[1], -1, dtype=torch.int32, device=DEV)[None].contiguous()
        far = pool[:, layers - 1]
        far[table[0].long()] = small.pages[small.table[0].long()]
        cache = pisa.PagedCache(far, table, page)
        q, start = normal(g, 1, 200, 8, 64), i32([n - 200])
        assert torch.equal(pisa.cache_prompt_attention(q, cache, start), pisa.cache_prompt_attention(q, small, start))
        a, b = (pisa.cache_attention(q[:, -1:], c, start + 200, window=900, cap=5.0) for c in (cache, small))
        assert torch.equal(a, b)
        del pool, far, cache


def test_far_positions_and_slopes():
    """A bias by distance at positions where its own size would drown the scores in 32 bits."""
    g = gen(13)
    page, at = 256, 120_000
    cache = make_cache(g, 1, at + 200, 1, page, 4)
    q = normal(g, 1, 150, 2, 64)
    s = torch.tensor([0.5, 3.0], device=DEV)
    got = pisa.cache_prompt_attention(q, cache, i32([at]), slopes=s)
    check(got, expected(q, cache, [at], [150], slopes=s))


def test_refusals():
    g = gen(14)
    cache = make_cache(g, 2, 40, 2, 16, 16)
    q, n = normal(g, 2, 20, 8, 64), i32([0, 5])
    for kw in (dict(first=torch.zeros(2, 19, dtype=torch.int32, device=DEV)), dict(last=torch.zeros(2, 20, device=DEV)),
               dict(out=torch.empty(2, 20, 8, 64, device=DEV)), dict(counts=i32([1])), dict(slopes=torch.zeros(9, device=DEV)),
               dict(window=-2), dict(first=torch.zeros(20, 2, dtype=torch.int32, device=DEV).t())):
        with pytest.raises(ValueError):
            pisa.cache_prompt_attention(q, cache, n, **kw)
    with pytest.raises(ValueError):
        pisa.cache_prompt_attention(q.float(), cache, n)
    for f in (lambda: pisa.cache_prompt_attention(q[:, :, :6], cache, n),
              lambda: pisa.cache_prompt_attention(q, cache, n, cap=-2.0),
              lambda: pisa.cache_prompt_attention(q, cache, n, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises(pisa.PisaError):
            f()


def test_past_the_tables_capacity():
    """Tokens past what the table holds: cut and flagged, and nothing else is read."""
    g = gen(15)
    cache = make_cache(g, 1, 128, 1, 64, 16)
    q = normal(g, 1, 100, 4, 64)
    ws = pisa.cache_workspace(cache)
    got = pisa.cache_prompt_attention(q, cache, i32([60]), workspace=ws)
    assert status(ws) == 6 and bool(torch.isfinite(got).all())
    whole = pisa.cache_prompt_attention(q[:, :68], cache, i32([60]))
    assert torch.equal(got[:, :68], whole)
