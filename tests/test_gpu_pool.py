"""Pages that sequences share: fork, reserve and compact against plain Python, and together with the cache's calls."""
import random

import pytest
import torch

import pool_ref
import pyramid_top_block_gb300 as pisa
from test_gpu_cache import DEV, gen, i32, normal, status

pytestmark = pytest.mark.gpu


def make_pool(r, B, wide, n_pages, page, held, words=4, spread=1):
    """A pool of small pages (each filled with a number of its own), sequences that hold held[b] pages, some shared."""
    pages = torch.arange(n_pages * spread, dtype=torch.int64, device=DEV)[:, None].expand(-1, words).contiguous()
    pages = pages.view(n_pages, spread, words)[:, 0]
    order = r.sample(range(n_pages), n_pages)
    table, refs, at = [], [0] * n_pages, 0
    for b in range(B):
        row = [-1] * wide
        for e in range(held[b]):
            if b and r.random() < 0.3 and table[b - 1][e] >= 0:
                row[e] = table[b - 1][e]
            else:
                row[e] = order[at]
                at += 1
            refs[row[e]] += 1
        table.append(row)
    lengths = [max(0, h * page - r.randrange(page)) for h in held]
    return pages, i32(table), i32(refs), i32(lengths)


def mirror(pages, table, refs, lengths, page):
    return pool_ref.Pool(table.tolist(), refs.tolist(), lengths.tolist(), page, [tuple(x) for x in pages.tolist()])


def same(m, pages, table, refs, lengths):
    assert table.tolist() == m.table
    assert refs.tolist() == m.refs
    assert lengths.tolist() == m.lengths
    assert [tuple(x) for x in pages.tolist()] == m.pages


def counted(table, n_pages):
    """References as the table has them."""
    x = table[(table >= 0) & (table < n_pages)].long()
    return torch.bincount(x, minlength=n_pages).tolist()


@pytest.mark.parametrize("B,wide,n_pages,page,words,spread", [
    (1, 1, 1, 16, 2, 1),
    (1, 5, 9, 64, 4, 2),
    (3, 7, 40, 32, 514, 1),
    (17, 33, 700, 16, 6, 3),
    (64, 70, 9000, 128, 2, 1),
    (130, 3, 500, 256, 4, 1),
    (300, 40, 20000, 64, 2, 1),
    (5, 2100, 12000, 16, 2, 1),
])
def test_a_run_of_calls(B, wide, n_pages, page, words, spread):
    """Forks, reserves, lengths that grow by what was granted, frees and compactions, all state compared each time."""
    r = random.Random(B * 1000 + wide)
    most = max(1, min(wide, n_pages * 2 // (3 * B)))
    held = [r.randrange(0, most + 1) for _ in range(B)]
    pages, table, refs, lengths = make_pool(r, B, wide, n_pages, page, held, words, spread)
    assert refs.tolist() == counted(table, n_pages)
    m = mirror(pages, table, refs, lengths, page)
    pool = pisa.PagePool(pages, table, refs, page)
    ws = pisa.pool_workspace(pool)
    flagged = False
    for step in range(12):
        kind = r.choice(["fork", "reserve", "reserve", "compact", "free"]) if step else "reserve"
        if kind in ("fork", "free"):
            parents = list(range(B))
            for b in range(B):
                if r.random() < (0.5 if kind == "fork" else 0.3):
                    parents[b] = r.randrange(B) if kind == "fork" else -1
            if step == 7:
                parents[r.randrange(B)] = B + r.randrange(3)
            flagged |= m.fork(parents)
            pisa.cache_fork(pool, i32(parents), lengths, workspace=ws)
        elif kind == "reserve":
            T = r.choice([1, 1, 3, page, 5 * page])
            counts = None if r.random() < 0.4 else [r.choice([0, T, r.randint(0, T), T + 5, -1]) for _ in range(B)]
            clipped = [T] * B if counts is None else [min(max(c, 0), T) for c in counts]
            granted, bad = m.reserve(clipped)
            flagged |= bad
            got = pisa.cache_reserve(pool, lengths, T, counts=None if counts is None else i32(counts), workspace=ws)
            assert got.tolist() == granted
            if r.random() < 0.7:  # the tokens are written
                lengths += got
                m.lengths = [n + c for n, c in zip(m.lengths, granted)]
        else:
            used = m.compact()
            assert int(pisa.cache_compact(pool, workspace=ws)) == used
        same(m, pages, table, refs, lengths)
        assert refs.tolist() == counted(table, n_pages)
        assert (status(ws) == 6) == flagged


def test_more_sequences_than_a_columns_chunk():
    """A fork of many sequences (few columns in a CTA), a table wider than one CTA's columns, and the most there are."""
    r = random.Random(1)
    for B, wide in ((2000, 45), (9000, 3), (32768, 2)):
        n_pages = B
        table = torch.randint(-1, n_pages, (B, wide), generator=gen(B), device=DEV, dtype=torch.int32)
        refs = i32(counted(table, n_pages))
        lengths = torch.randint(0, 16 * wide, (B,), generator=gen(2), device=DEV, dtype=torch.int32)
        parents = torch.randint(-1, B, (B,), generator=gen(3), device=DEV, dtype=torch.int32)
        q = parents.long()
        want = torch.where(q[:, None] >= 0, table[q.clamp(min=0)], -1)
        want_n = torch.where(q >= 0, lengths[q.clamp(min=0)], 0)
        pool = pisa.PagePool(torch.zeros(n_pages, 16, dtype=torch.uint8, device=DEV), table, refs, 16)
        pisa.cache_fork(pool, parents, lengths)
        assert torch.equal(table, want) and torch.equal(lengths, want_n) and refs.tolist() == counted(want, n_pages)
    pool = pisa.PagePool(torch.zeros(4, 16, dtype=torch.uint8, device=DEV), i32([[-1]] * 32769), i32([0] * 4), 16)
    with pytest.raises(pisa.PisaError):
        pisa.cache_fork(pool, i32([0] * 32769), i32([0] * 32769))


def test_a_lack_of_pages():
    """Sequences are served in order; the first that finds too few pages, and those after it that need any, stay as they
    are, and the pages that a call lets go are there for the next one."""
    page = 16
    table = i32([[0, -1, -1], [0, -1, -1], [1, 2, -1], [-1, -1, -1]])
    refs = i32([2, 1, 1, 0, 0])
    lengths = i32([5, 5, 20, 0])
    pages = torch.arange(5, dtype=torch.int64, device=DEV)[:, None].expand(5, 2).contiguous()
    pool = pisa.PagePool(pages, table, refs, page)
    m = mirror(pages, table, refs, lengths, page)
    # 0 and 1 replace their shared page, 2 writes into its own, 3 would need a page that 0 and 1 let go only now
    for counts in ([1, 1, 1, 1], [1, 1, 1, 1], [0, 0, 12, 40], [0, 0, 13, 1], [0, 0, 0, 16]):
        want = m.reserve(counts)[0]
        assert pisa.cache_reserve(pool, lengths, 40, counts=i32(counts)).tolist() == want
        same(m, pages, table, refs, lengths)
    assert want == [0, 0, 0, 16]


def test_lengths_out_of_range():
    table, refs = i32([[-1, -1]] * 4), i32([0] * 9)
    lengths = i32([-1, 32, 31, (1 << 31) - 1])
    pages = torch.zeros(9, 2, dtype=torch.int64, device=DEV)
    pool = pisa.PagePool(pages, table, refs, 16)
    ws = pisa.pool_workspace(pool)
    m = mirror(pages, table, refs, lengths, 16)
    want, bad = m.reserve([1] * 4)
    assert bad and pisa.cache_reserve(pool, lengths, 1, workspace=ws).tolist() == want == [0, 0, 1, 0]
    same(m, pages, table, refs, lengths)
    assert status(ws) == 6


@pytest.mark.parametrize("bits,layers", [(16, 1), (4, 2)])
def test_samples_of_one_prompt(bits, layers):
    """A prompt, four samples of it that go apart, one freed, the pool compacted: every sample attends as a cache of
    its own would, eagerly and by a graph of the same steps."""
    g = gen(21)
    B, Hq, Hkv, page, n0, steps = 5, 8, 2, 16, 37, 3

    def fresh():
        p = pisa.PagePool.allocate(B, 120, Hkv, 60, page, bits, layers)
        return p, torch.zeros(B, dtype=torch.int32, device=DEV), pisa.pool_workspace(p), pisa.cache_workspace(p.layer())

    rotary = pisa.rotary_table(128)
    prompt = [normal(g, B, n0, h, 64) for h in (Hq, Hkv, Hkv)]
    news = [[normal(g, B, 1, h, 64) for h in (Hq, Hkv, Hkv)] for _ in range(2 * steps)]
    only = i32([n0, 0, 0, 0, 0])
    parents, free = i32([0, 0, 0, 0, -1]), i32([0, -1, 2, 2, -1])

    def run(p, lengths, pws, cws, graph):
        caches = [p.layer(i) for i in range(layers)]
        outs = []
        got = pisa.cache_reserve(p, lengths, n0, counts=only, workspace=pws)
        for c in caches:
            q, _ = pisa.cache_append(*prompt, c, lengths, rotary, counts=got, workspace=cws)
        outs.append(pisa.cache_prompt_attention(q, caches[-1], lengths, counts=got, workspace=cws, out=torch.zeros_like(q)))
        lengths += got
        pisa.cache_fork(p, parents, lengths, workspace=pws)
        alive = i32([1, 1, 1, 1, 0])
        tokens = [[x.clone() for x in news[0]]]

        def step(x, c_new):
            got = pisa.cache_reserve(p, lengths, 1, counts=c_new, workspace=pws)
            for c in caches:
                q, _ = pisa.cache_append(*x, c, lengths, rotary, counts=got, workspace=cws)
            lengths.add_(got)
            return pisa.cache_attention(q, caches[-1], lengths, workspace=cws, window=30)

        if graph:
            x = tokens[0]
            state = [t.clone() for t in (p.table, p.refs, lengths, p.pages)]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step(x, alive)
            torch.cuda.current_stream().wait_stream(side)
            for t, was in zip((p.table, p.refs, lengths, p.pages), state):
                t.copy_(was)
            cg = torch.cuda.CUDAGraph()
            with torch.cuda.graph(cg):
                out = step(x, alive)
        for i in range(2 * steps):
            if i == steps:
                pisa.cache_fork(p, free, lengths, workspace=pws)
                pisa.cache_compact(p, workspace=pws)
                alive.copy_(i32([1, 0, 1, 1, 0]))
            if graph:
                for dst, src in zip(x, news[i]):
                    dst.copy_(src)
                cg.replay()
                outs.append(out.clone())
            else:
                outs.append(step(news[i], alive))
        assert status(pws) == 0 and status(cws) == 0
        assert p.refs.tolist() == counted(p.table, p.n_pages)
        return outs, lengths

    a, n = run(*fresh(), False)
    b, n2 = run(*fresh(), True)
    assert torch.equal(n, n2)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    # the same by caches of their own: each sample's tokens one after the other, no page shared
    def alone(plan):  # plan: (sample that wrote, step) of each decoding step of the path
        c = pisa.PagedCache.allocate(1, 120, Hkv, page, bits)
        zero = i32([0])
        pisa.cache_append(*[x[:1] for x in prompt], c, zero, rotary)
        out = None
        for i, (s, t) in enumerate(plan):
            at = i32([n0 + i])
            q, _ = pisa.cache_append(*[x[s:s + 1] for x in news[t]], c, at, rotary)
            out = pisa.cache_attention(q, c, at + 1, window=30)
        return out

    for s in (0, 1, 2, 3):
        for i in range(steps):
            assert torch.equal(a[1 + i][s:s + 1], alone([(s, t) for t in range(i + 1)])), (s, i)
    for s, parent in ((0, 0), (2, 2), (3, 2)):  # sample 3 went on from sample 2
        path = [(parent, t) for t in range(steps)] + [(s, t) for t in range(steps, 2 * steps)]
        assert torch.equal(a[2 * steps][s:s + 1], alone(path)), s


def test_on_another_stream():
    """Calls on a stream of their own, and between streams that wait for one another."""
    r = random.Random(5)
    pages, table, refs, lengths = make_pool(r, 20, 9, 300, 16, [r.randrange(8) for _ in range(20)], words=2000)
    m = mirror(pages, table, refs, lengths, 16)
    pool = pisa.PagePool(pages, table, refs, 16)
    ws = pisa.pool_workspace(pool)
    parents = [r.randrange(-1, 20) for _ in range(20)]
    s = torch.cuda.Stream()
    par = i32(parents)
    s.wait_stream(torch.cuda.current_stream())
    m.fork(parents)
    pisa.cache_fork(pool, par, lengths, workspace=ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    want = m.reserve([3] * 20)[0]
    got = pisa.cache_reserve(pool, lengths, 3, workspace=ws)
    s.wait_stream(torch.cuda.current_stream())
    used = pisa.cache_compact(pool, workspace=ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert got.tolist() == want and int(used) == m.compact()
    same(m, pages, table, refs, lengths)


def test_refusals():
    pages, table, refs = torch.zeros(4, 8, dtype=torch.int64, device=DEV), i32([[-1, -1]] * 2), i32([0] * 4)
    for args in ((pages, table, refs, 20), (pages[:, ::2], table, refs, 16), (pages[:, :1], table, refs, 16),
                 (pages, table.long(), refs, 16), (pages, table, refs[:3], 16), (pages.cpu(), table, refs, 16)):
        with pytest.raises(ValueError):
            pisa.PagePool(*args)
    pool = pisa.PagePool(pages, table, refs, 16)
    n = i32([0, 0])
    for f in (lambda: pisa.cache_fork(pool, i32([0]), n), lambda: pisa.cache_fork(pool, n.long(), n),
              lambda: pisa.cache_reserve(pool, n, 1, counts=i32([1])), lambda: pisa.cache_reserve(pool, n[:1], 1),
              lambda: pisa.cache_reserve(pool, n, 1, granted=torch.zeros(2, device=DEV)),
              lambda: pisa.cache_compact(pool, used=i32([0, 0]))):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: pisa.cache_reserve(pool, n, 0),
              lambda: pisa.cache_compact(pool, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(pisa.PisaError):
            f()
