"""The cache calls on several streams that wait for one another, eagerly and captured into one graph."""
import pytest
import torch

import pyramid_top_block_gb300 as pisa
import test_gpu_cache as base

pytestmark = pytest.mark.gpu
DEV = base.DEV


@pytest.mark.parametrize("bits", [16, 4])
def test_two_branches_that_meet(bits):
    """A step whose two attention calls run on two streams, each with its own workspace, between an append that both
    wait for and another that waits for both (it overwrites what they read)."""
    B, Hq, Hkv, n, steps = 3, 16, 2, 6000, 6
    g = base.gen(50 + bits)
    cache = base.make_cache(g, B, n + 70, Hkv, 64, bits)
    first = cache.pages.clone()
    rotary = pisa.rotary_table(n + 70)
    new = [[base.normal(g, B, 40, h, 64) for h in (Hq, Hkv, Hkv)] for _ in range(steps)]
    x = [t.clone() for t in new[0]]
    start, lengths = base.i32([n, n - 1000, 5]), base.i32([n + 40, n - 960, 45])
    idx = torch.randint(0, 90, (B, Hkv, 8, 7), generator=g, device=DEV, dtype=torch.int32)
    side, ws = torch.cuda.Stream(), [pisa.cache_workspace(cache) for _ in range(2)]
    a, b = torch.cuda.Event(), torch.cuda.Event()
    outs = [torch.empty(B, 8, Hq, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    q_out, k_out = torch.empty_like(x[0]), torch.empty_like(x[1])
    k_read, v_read = torch.empty_like(x[1]), torch.empty_like(x[1])

    def step(two):
        pisa.cache_append(*x, cache, start, rotary, q_out=q_out, k_out=k_out)
        q = q_out[:, 32:]
        if two:
            a.record()
            side.wait_event(a)
        pisa.cache_attention(q, cache, lengths, out=outs[0], workspace=ws[0])
        pisa.cache_attention(q, cache, lengths, idx=idx, out=outs[1], workspace=ws[1], stream=side if two else None)
        if two:
            b.record(side)
            torch.cuda.current_stream().wait_event(b)
        pisa.cache_append(None, x[2], x[1], cache, start, None, k_out=k_out)
        pisa.cache_read(cache, start, 40, k_out=k_read, v_out=v_read)

    def run(make):
        cache.pages.copy_(first)
        got = []
        for s in range(steps):
            for dst, src in zip(x, new[s]):
                dst.copy_(src)
            make()
            got.append([t.clone() for t in (*outs, k_out, k_read, v_read, cache.pages)])
        torch.cuda.synchronize()
        return got

    want = run(lambda: step(False))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(True)
    for make in (lambda: step(True), graph.replay):
        for s, (w, h) in enumerate(zip(want, run(make))):
            for i, (p, q) in enumerate(zip(w, h)):
                assert torch.equal(p, q), (s, i)
    assert base.status(ws[0]) == 0 and base.status(ws[1]) == 0


@pytest.mark.parametrize("bits", [16, 4])
def test_a_call_for_very_many_sequences(bits):
    """As many sequences as a cache may have, over shared pages; some empty."""
    B = 65535
    g = base.gen(60)
    short = base.make_cache(g, 5, 200, 1, 64, bits)
    which = torch.arange(B, device=DEV) % 5
    for cache in (pisa.PagedCache(short.pages, short.table[which].contiguous(), 64),
                  base.in_a_wide_table(pisa.PagedCache(short.pages, short.table[which].contiguous(), 64), 2100)):
        n = [0, 200, 64, 1, 130]
        lengths = torch.tensor(n, dtype=torch.int32, device=DEV)[which].contiguous()
        q = base.normal(g, 5, 1, 2, 64)
        out = torch.full((B, 1, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        ws = pisa.cache_workspace(cache)
        pisa.cache_attention(q[which].contiguous(), cache, lengths, out=out, workspace=ws)
        assert base.status(ws) == 0
        some = out[:5]
        base.check_attention(short, q, n, some)
        for b in range(5):  # (in the stream a unit may be cut, which changes sums)
            rows = out[which == b].float()
            assert bool(((rows - some[b].float()).abs() <= 2.0 ** -7 * some[b].float().abs() + 2.0 ** -9).all())
        k, v = pisa.cache_read(cache, torch.zeros(B, dtype=torch.int32, device=DEV), 2, counts=lengths.clamp(max=2))
        kk, vv = pisa.cache_read(short, torch.zeros(5, dtype=torch.int32, device=DEV), 2)
        assert torch.equal(k[which == 1], kk[1:2].expand_as(k[which == 1]))
        assert torch.equal(v[which == 4], vv[4:5].expand_as(v[which == 4]))
