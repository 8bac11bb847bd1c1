"""The paged KV cache on the GPU: append with rotation, attention over it, reading it back, against 64 bits."""
import pytest
import torch

import cache_ref as ref
import pyramid_top_block_gb300 as pisa

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)


def make_cache(g, B, n_cap, Hkv, page, bits, k_exp=0, v_exp=0, fill=True, extra=3, layers=1):
    """A cache whose pages are shuffled over a pool (of `layers` interleaved layers) and filled with noise."""
    per = -(-n_cap // page)
    n = B * per + extra
    U = min(page, 64)
    inner = (2, U, 64) if bits == 16 else (72 * U,)
    shape = (n, layers, Hkv, page // U) + inner
    if bits == 16:
        pool = torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)
    else:
        pool = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
        for base in (32, 68):  # scales from about 1/32 to 4
            s = pool[..., base * U:(base + 4) * U]
            s.copy_(torch.randint(16, 73, s.shape, generator=g, device=DEV, dtype=torch.uint8))
    if not fill:
        pool.zero_()
    table = torch.randperm(n, generator=g, device=DEV)[:B * per].view(B, per).to(torch.int32)
    return pisa.PagedCache(pool[:, layers // 2], table, page, k_exp, v_exp)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def status(ws):
    return pisa.check_device_status(ws)


# ------------------------------------------------------------------------------------------ append and read


def check_append(cache, q, k, v, start, counts, rotary, interleaved, q_out, k_out, before):
    """Every output bit: the rotated rows, the pages of the appended tokens, and everything else as before."""
    B, T = k.shape[:2]
    want = {}
    for b in range(B):
        for t in range(min(T, counts[b])):
            p = start[b] + t
            kk, qq = k[b, t].double(), None if q is None else q[b, t].double()
            if rotary is not None:
                pos = torch.tensor(p, device=DEV)
                kk = ref.rotate(k[b, t], rotary, pos, interleaved)
                qq = None if q is None else ref.rotate(q[b, t], rotary, pos, interleaved)
            kk = ref.to_bf16(kk)
            assert torch.equal(k_out[b, t], kk), (b, t)
            if q is not None:
                assert torch.equal(q_out[b, t], ref.to_bf16(qq)), (b, t)
            want[b, p] = (kk, v[b, t])
    U = min(cache.page_size, 64)
    expect = before.clone()
    for (b, p), kv in want.items():
        page, rec, u = int(cache.table[b, p // cache.page_size]), (p % cache.page_size) // U, p % U
        for i in range(2):
            if cache.bits == 16:
                expect[page, :, rec, i, u] = kv[i]
            else:
                c, s = ref.quantise(kv[i].double(), (cache._struct.k_exp, cache._struct.v_exp)[i])
                code = torch.searchsorted(ref.E2M1.to(DEV), c.abs().contiguous()).to(torch.uint8)
                code |= (c < 0).to(torch.uint8) << 3
                expect[page, :, rec, 36 * U * i + 32 * u:36 * U * i + 32 * (u + 1)] = code[..., 0::2] | code[..., 1::2] << 4
                expect[page, :, rec, 36 * U * i + 32 * U + 4 * u:36 * U * i + 32 * U + 4 * (u + 1)] = s
    got = cache.pages
    if cache.bits == 4:  # a zero may be held with either sign
        def plain(x):
            x = x.clone()
            for i in range(2):
                c = x[..., 36 * U * i:36 * U * i + 32 * U]
                c.copy_(torch.where(c & 15 == 8, c - 8, c))
                c.copy_(torch.where(c >> 4 == 8, c - 128, c))
            return x
        expect, got = plain(expect), plain(got)
    assert torch.equal(got, expect)


@pytest.mark.parametrize("B,T,Hq,Hkv,page,bits,rot,interleaved", [
    (1, 1, 32, 2, 64, 4, 64, False),
    (3, 1, 16, 16, 16, 16, 64, True),
    (2, 5, 8, 1, 32, 4, 32, True),
    (2, 70, 4, 2, 128, 16, 48, False),
    (1, 133, 6 * 2, 6, 256, 4, 16, False),
    (2, 33, 32, 2, 16, 4, 48, True),
    (4, 3, 8, 8, 64, 16, 0, False),
])
def test_append(B, T, Hq, Hkv, page, bits, rot, interleaved):
    g = gen(B * 1000 + T)
    cap = T + 90
    cache = make_cache(g, B, cap, Hkv, page, bits, layers=2, k_exp=1 if bits == 4 else 0, v_exp=-2 if bits == 4 else 0)
    qkv = normal(g, B, T, Hq + 2 * Hkv, 64)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 2)
    start = [(7 * b + 61) % 90 for b in range(B)]
    counts = [max(0, T - 2 * b) for b in range(B)]
    rotary = pisa.rotary_table(cap, rot) if rot else None
    before = cache.pages.clone()
    q_out, k_out = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    ws = pisa.cache_workspace(cache)
    pisa.cache_append(q, k, v, cache, i32(start), rotary, counts=i32(counts), interleaved=interleaved, q_out=q_out,
                      k_out=k_out, workspace=ws)
    assert status(ws) == 0
    check_append(cache, q, k, v, start, counts, rotary, interleaved, q_out, k_out, before)
    for b in range(B):  # rows behind a sequence's count stay as they were
        assert bool((q_out[b, counts[b]:] == 7).all()) and bool((k_out[b, counts[b]:] == 7).all())


def test_append_in_place_and_allocated_outputs():
    g = gen(5)
    cache = make_cache(g, 2, 40, 2, 16, 16)
    q, k, v = normal(g, 2, 9, 8, 64), normal(g, 2, 9, 2, 64), normal(g, 2, 9, 2, 64)
    rotary = pisa.rotary_table(40)
    start = i32([0, 20])
    qo, ko = pisa.cache_append(q, k, v, cache, start, rotary)
    first = cache.pages.clone()
    q2, k2 = q.clone(), k.clone()
    a, b = pisa.cache_append(q2, k2, v, cache, start, rotary, q_out=q2, k_out=k2)
    assert a is q2 and b is k2 and torch.equal(q2, qo) and torch.equal(k2, ko)
    assert torch.equal(first, cache.pages)
    none, k3 = pisa.cache_append(None, k, v, cache, start, rotary)
    assert none is None and torch.equal(k3, ko) and torch.equal(first, cache.pages)


def test_append_a_prompt_equals_token_by_token():
    """The bits of a token do not depend on the call that appended it."""
    g = gen(6)
    q, k, v = normal(g, 1, 200, 4, 64), normal(g, 1, 200, 2, 64), normal(g, 1, 200, 2, 64)
    rotary = pisa.rotary_table(100000)[-300:].contiguous()
    a, b = make_cache(gen(1), 1, 300, 2, 64, 4, fill=False), make_cache(gen(1), 1, 300, 2, 64, 4, fill=False)
    qa, ka = pisa.cache_append(q, k, v, a, i32([50]), rotary)
    for t in range(200):
        qb, kb = pisa.cache_append(q[:, t:t + 1], k[:, t:t + 1], v[:, t:t + 1], b, i32([50 + t]), rotary)
        assert torch.equal(qb[:, 0], qa[:, t]) and torch.equal(kb[:, 0], ka[:, t])
    assert torch.equal(a.pages, b.pages)


def special_rows():
    """Rows at and next to the format's borders: ties of codes and scales, zeros, subnormals, large, not finite."""
    rows = []
    for m in range(8, 16):  # scales of every mantissa, values on and next to every border
        for e in (-6, 0, 5):
            s = m * 2.0 ** (e - 3)
            x = [6 * s, -6 * s]
            for c in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
                x += [c * s, -c * s]
            rows.append(x * 4)
    for top in (0.0, 2.0 ** -133, 6 * 2.0 ** -10, 1.01 * 6 * 2.0 ** -10, 6 * 2.0 ** -9, 9 * 2.0 ** -9, 2688.0, 2800.0,
                1e30, 3.3e38):
        rows.append([top, -top / 2, top / 3, top / 5] * 16)
    x = torch.tensor(rows, dtype=torch.float64, device=DEV).float().to(torch.bfloat16)
    bits = x.view(torch.int16)
    near = torch.cat([x, (bits + 1).view(torch.bfloat16), (bits - 1).view(torch.bfloat16)])
    near = near.clone()
    near[5, 3], near[6, 20], near[7, 63] = float("inf"), NAN, float("-inf")
    return near


def test_append_borders_of_the_4_bit_format():
    x = special_rows()
    n = x.shape[0]
    for k_exp in (0, -5, 24):
        cache = make_cache(gen(2), 1, n, 1, 64, 4, k_exp=k_exp, v_exp=-3)
        k, v = x.view(1, n, 1, 64), x.flip(0).reshape(1, n, 1, 64)
        _, k_out = pisa.cache_append(None, k, v, cache, i32([0]), None)
        assert torch.equal(k_out.view(torch.int16), k.view(torch.int16))
        got = ref.tokens(cache, 0, n)
        kr, vr = pisa.cache_read(cache, i32([0]), n)
        for i, (y, exp) in enumerate(((k, k_exp), (v, -3))):
            c, s = ref.quantise(y[0].double(), exp)
            torch.testing.assert_close(got[i], ref.values(c, s, exp), rtol=0, atol=0, equal_nan=True)
            r = (kr, vr)[i][0].double()
            torch.testing.assert_close(r, got[i], rtol=0, atol=0, equal_nan=True)


def test_append_rotation_of_special_values():
    """Cancellation, subnormals, infinities and exact ties of the rotation's rounding."""
    n = 64
    g = gen(3)
    k = normal(g, 1, n, 1, 64)
    k[0, 0, 0, 32:] = k[0, 0, 0, :32]           # equal halves at 45 degrees: exact zeros
    k[0, 1] *= 2.0 ** -120
    k[0, 2, 0, 5] = float("inf")
    k[0, 3, 0, 40] = NAN
    k[0, 4] *= 2.0 ** 100
    rotary = pisa.rotary_table(n)
    rotary[0] = 0.5 ** 0.5
    rotary[5, :32], rotary[5, 32:] = 1 + 2.0 ** -8, 0.0  # half a step above, with x of 8 bits: ties
    rotary[6, :32], rotary[6, 32:] = 1 + 2.0 ** -8, 2.0 ** -60
    cache = make_cache(g, 1, n, 1, 64, 16)
    _, ko = pisa.cache_append(None, k, k, cache, i32([0]), rotary)
    pos = torch.arange(n, device=DEV)
    want = ref.to_bf16(ref.rotate(k[0], rotary, pos, False))
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(ko[0]), torch.isnan(want))
    assert torch.equal(ko[0][fin], want[fin])


@pytest.mark.parametrize("bits", [16, 4])
def test_append_out_of_range_is_left_out(bits):
    g = gen(8)
    cache = make_cache(g, 4, 32, 2, 16, bits)
    cache.table[1, 1] = cache.n_pages
    cache.table[2, 0] = -1
    q, k, v = normal(g, 4, 20, 4, 64), normal(g, 4, 20, 2, 64), normal(g, 4, 20, 2, 64)
    before = cache.pages.clone()
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    ws = pisa.cache_workspace(cache)
    start = [20, 2, -3, 3]   # past the end; into a bad page; negative, then a bad page; past the table of angles
    rotary = pisa.rotary_table(21)
    pisa.cache_append(q, k, v, cache, i32(start), rotary, q_out=qo, k_out=ko, workspace=ws)
    assert status(ws) == 6
    keep = {0: [20], 1: range(2, 16), 2: range(16, 17), 3: range(3, 21)}
    at = {(b, p) for b, ps in keep.items() for p in ps}
    U = 16
    expect = before.clone()
    for b in range(4):
        for t in range(20):
            p = start[b] + t
            if (b, p) in at:
                assert torch.equal(ko[b, t], ref.to_bf16(ref.rotate(k[b, t], rotary, torch.tensor(p, device=DEV), False)))
                page = int(cache.table[b, p // 16])
                if bits == 16:
                    expect[page, :, 0, 0, p % 16], expect[page, :, 0, 1, p % 16] = ko[b, t], v[b, t]
                else:
                    for i in range(2):
                        for lo, w in ((36 * U * i + 32 * (p % 16), 32), (36 * U * i + 32 * U + 4 * (p % 16), 4)):
                            expect[page, :, 0, lo:lo + w] = cache.pages[page, :, 0, lo:lo + w]
            else:
                assert bool((ko[b, t] == 7).all()) and bool((qo[b, t] == 7).all()), (b, t)
    assert torch.equal(cache.pages, expect)


@pytest.mark.parametrize("B,T,Hkv,page,bits", [(1, 1, 1, 64, 4), (3, 77, 2, 16, 16), (2, 300, 4, 256, 4), (2, 31, 32, 32, 16)])
def test_read(B, T, Hkv, page, bits):
    g = gen(T)
    cache = make_cache(g, B, T + 50, Hkv, page, bits, layers=3, k_exp=3 if bits == 4 else 0, v_exp=-24 if bits == 4 else 0)
    start, counts = [(17 * b + 3) % 50 for b in range(B)], [max(0, T - 5 * b) for b in range(B)]
    wide = torch.full((B, T, 2 * Hkv + 1, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    k, v = wide[:, :, :Hkv], wide[:, :, Hkv + 1:]
    pisa.cache_read(cache, i32(start), T, counts=i32(counts), k_out=k, v_out=v)
    for b in range(B):
        kk, vv = ref.tokens(cache, b, start[b] + counts[b])
        m = counts[b]
        assert torch.equal(k[b, :m].double(), kk[start[b]:]) and torch.equal(v[b, :m].double(), vv[start[b]:])
        assert bool((wide[b, m:] == 7).all()) and bool((wide[b, :, Hkv] == 7).all())


def test_read_bad_pages_are_left_out():
    g = gen(9)
    cache = make_cache(g, 1, 64, 1, 16, 16)
    cache.table[0, 1] = -5
    cache.table[0, 2] = 1 << 30
    ws = pisa.cache_workspace(cache)
    k = torch.full((1, 80, 1, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    pisa.cache_read(cache, i32([-8]), 80, k_out=k, v_out=v, workspace=ws)
    assert status(ws) == 6
    seen = torch.zeros(80, dtype=torch.bool, device=DEV)
    seen[8:24] = True    # positions 0 .. 15
    seen[56:72] = True   # positions 48 .. 63
    assert bool((k[0, ~seen] == 7).all()) and not bool((k[0, seen] == 7).all(-1).any())


# ------------------------------------------------------------------------------------------------ attention


def check_attention(cache, q, lengths, out, idx=None, rows=None):
    """out against 64 bits on the values that the cache holds."""
    B, T, Hq, _ = q.shape
    G = Hq // cache.Hkv
    for b in range(B):
        n = lengths[b]
        k, v = ref.tokens(cache, b, max(n, 1))
        for t in range(T):
            if rows is not None and (b, t) not in rows:
                continue
            see = n - T + t + 1
            for h in range(cache.Hkv):
                o = out[b, t, h * G:(h + 1) * G].double()
                if see <= 0:
                    assert bool((o == 0).all()), (b, t, h)
                    continue
                if idx is None:
                    keep = torch.ones(see, dtype=torch.int64, device=DEV)
                else:
                    keep = torch.zeros(see, dtype=torch.int64, device=DEV)
                    for blk in idx[b, h, t].tolist():
                        if 0 <= blk * 64 < see:
                            keep[blk * 64:blk * 64 + 64] += 1
                want, pv, sv, big = ref.attention(q[b, t, h * G:(h + 1) * G].double(), k[:see, h], v[:see, h], keep)
                tol = ref.tolerance(want, pv, sv, big, see, cache.bits, out.dtype)
                err = (o - want).abs()
                assert bool((err <= tol).all()), (b, t, h, float((err / tol.clamp(min=1e-300)).max()))


ALL = [
    # B, T, G, Hkv, page, lengths
    (1, 1, 16, 2, 64, [1]),
    (1, 1, 1, 1, 16, [64]),
    (3, 1, 16, 2, 64, [65, 0, 300]),
    (2, 1, 4, 8, 128, [1000, 129]),
    (4, 3, 4, 2, 32, [1201, 2, 64, 66]),
    (2, 16, 16, 1, 256, [700, 5]),
    (2, 16, 1, 2, 16, [260, 16]),
    (3, 5, 2, 3, 16, [63, 128, 513]),
    (40, 1, 8, 2, 64, [(37 * b) % 211 for b in range(40)]),
    (1, 2, 8, 2, 64, [20011]),
    (2, 1, 16, 2, 16, [9000, 12345]),
]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("B,T,G,Hkv,page,lengths", ALL)
def test_attention_over_all(bits, B, T, G, Hkv, page, lengths):
    g = gen(B * 100 + T)
    cache = make_cache(g, B, max(lengths) + 40, Hkv, page, bits, layers=2)
    q = normal(g, B, T, G * Hkv + 3, 64)[:, :, 3:]  # rows of a wider tensor
    ws = pisa.cache_workspace(cache)
    out = pisa.cache_attention(q, cache, i32(lengths), workspace=ws)
    assert out.dtype == torch.bfloat16 and status(ws) == 0
    check_attention(cache, q, lengths, out)
    o32 = torch.empty(out.shape, dtype=torch.float32, device=DEV)
    pisa.cache_attention(q, cache, i32(lengths), out=o32, workspace=ws)
    check_attention(cache, q, lengths, o32)
    again = pisa.cache_attention(q, cache, i32(lengths), workspace=ws)
    assert torch.equal(again, out)  # the same bits in every call


def listed_blocks(g, B, Hkv, T, K, lengths):
    M = max(2, -(-max(lengths) // 64) + 1)
    idx = torch.randint(-1, M, (B, Hkv, T, K), generator=g, device=DEV, dtype=torch.int32)
    idx[0, 0, 0, :] = -1                      # nothing listed
    if K > 1:
        idx[-1, -1, -1, 1] = idx[-1, -1, -1, 0]  # the same block twice
    return idx


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("B,T,G,Hkv,page,K,lengths", [
    (2, 1, 16, 2, 64, 8, [1000, 777]),
    (1, 1, 1, 1, 16, 1, [5]),
    (3, 2, 4, 2, 32, 3, [200, 0, 64]),
    (2, 5, 8, 1, 256, 32, [2500, 300]),
    (2, 16, 2, 2, 128, 64, [5000, 20]),
    (5, 1, 16, 4, 16, 9, [64, 65, 127, 128, 1]),
])
def test_attention_over_blocks(bits, B, T, G, Hkv, page, K, lengths):
    g = gen(B * 100 + K)
    cache = make_cache(g, B, max(lengths) + 40, Hkv, page, bits)
    q = normal(g, B, T, G * Hkv, 64)
    idx = listed_blocks(g, B, Hkv, T, K, lengths)
    ws = pisa.cache_workspace(cache)
    out = pisa.cache_attention(q, cache, i32(lengths), idx=idx, workspace=ws)
    assert status(ws) == 0
    check_attention(cache, q, lengths, out, idx=idx)
    o32 = torch.empty(out.shape, dtype=torch.float32, device=DEV)
    pisa.cache_attention(q, cache, i32(lengths), idx=idx, out=o32, workspace=ws)
    check_attention(cache, q, lengths, o32, idx=idx)
    if T == 1:
        assert torch.equal(pisa.cache_attention(q, cache, i32(lengths), idx=idx[:, :, 0].contiguous()), out)


@pytest.mark.parametrize("bits", [16, 4])
def test_blocks_in_order_equal_all(bits):
    """Every block listed is the whole cache."""
    g = gen(4)
    cache = make_cache(g, 2, 640, 2, 64, bits)
    q = normal(g, 2, 1, 32, 64)
    lengths = [640, 601]
    idx = torch.arange(10, device=DEV, dtype=torch.int32).expand(2, 2, 1, 10).contiguous()
    out = pisa.cache_attention(q, cache, i32(lengths), idx=idx)
    check_attention(cache, q, lengths, out)


def poison(cache, b, p, what="kv"):
    """NaNs (bf16: also infinities) for the token at position p of sequence b."""
    U = min(cache.page_size, 64)
    page, rec, u = int(cache.table[b, p // cache.page_size]), (p % cache.page_size) // U, p % U
    for i, name in enumerate("kv"):
        if name in what:
            if cache.bits == 16:
                cache.pages[page, :, rec, i, u] = NAN
                cache.pages[page, :, rec, i, u, ::3] = float("inf")
            else:
                cache.pages[page, :, rec, 36 * U * i + 32 * U + 4 * u:36 * U * i + 32 * U + 4 * u + 4] = 127


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("T,G,page,n", [(1, 16, 64, 100), (4, 4, 16, 130), (6, 1, 32, 66), (3, 16, 128, 65)])
def test_what_a_query_does_not_see_does_not_matter(bits, T, G, page, n):
    g = gen(n)
    cache = make_cache(g, 2, 256, 2, page, bits)
    q = normal(g, 2, T, 2 * G, 64)
    lengths = [n, n - 1]
    for b in range(2):
        for p in range(lengths[b], 256):
            poison(cache, b, p)
    cache.table[:, -(-n // page):] = -1  # pages that hold no token yet
    ws = pisa.cache_workspace(cache)
    out = pisa.cache_attention(q, cache, i32(lengths), workspace=ws)
    assert status(ws) == 0
    check_attention(cache, q, lengths, out)
    idx = torch.arange(-(-n // 64) + 1, device=DEV, dtype=torch.int32)
    idx = idx.expand(2, 2, T, idx.numel()).contiguous()
    out = pisa.cache_attention(q, cache, i32(lengths), idx=idx, workspace=ws)
    assert status(ws) == 0
    check_attention(cache, q, lengths, out)
    # the newest token's values are NaN: only its own query sees them
    for what in ("k", "v"):
        for b in range(2):
            poison(cache, b, lengths[b] - 1, what)
        for use in (None, idx):
            out = pisa.cache_attention(q, cache, i32(lengths), idx=use)
            check_attention(cache, q, lengths, out, rows={(b, t) for b in range(2) for t in range(T - 1)})
            assert bool(torch.isnan(out[:, T - 1]).any(-1).all())


@pytest.mark.parametrize("bits", [16, 4])
def test_bad_pages_give_nan_and_a_status(bits):
    g = gen(11)
    cache = make_cache(g, 3, 2000, 2, 64, bits)
    q = normal(g, 3, 1, 32, 64)
    lengths = [2000, 1500, 130]
    cache.table[1, 20] = cache.n_pages
    cache.table[2, 1] = -7
    ws = pisa.cache_workspace(cache)
    out = pisa.cache_attention(q, cache, i32(lengths), workspace=ws)
    assert status(ws) == 6
    assert bool(torch.isnan(out[1:]).all())
    good = pisa.PagedCache(cache.pages, cache.table[:1].contiguous(), 64)
    check_attention(good, q[:1], lengths[:1], out[:1])
    idx = i32([[[[0, 3]], [[0, 3]]], [[[0, 20]], [[0, 3]]], [[[0, -1]], [[1, 0]]]])
    ws = pisa.cache_workspace(cache)
    out = pisa.cache_attention(q, cache, i32(lengths), idx=idx, workspace=ws)
    assert status(ws) == 6
    nan = torch.isnan(out[:, 0]).all(-1).view(3, 2, 16).all(-1)
    assert nan.tolist() == [[False, False], [True, False], [False, True]]
    # a length past the table is cut to it, and flagged
    ws = pisa.cache_workspace(good)
    long = pisa.cache_attention(q[:1], good, i32([1 << 30]), workspace=ws)
    assert status(ws) == 6
    assert torch.equal(long, pisa.cache_attention(q[:1], good, i32([good.max_pages * 64])))
    assert bool((pisa.cache_attention(q[:1], good, i32([-5])) == 0).all())


@pytest.mark.parametrize("bits", [16, 4])
def test_large_and_small_queries_and_peaks(bits):
    """One key far above the rest, rows of very different sizes, zero rows."""
    g = gen(12)
    cache = make_cache(g, 1, 3000, 1, 64, bits)
    q = normal(g, 1, 1, 16, 64)
    q[0, 0, 0] *= 1000
    q[0, 0, 1] *= 2.0 ** -30
    q[0, 0, 2] = 0
    q[0, 0, 3, 1:] = 0
    q[0, 0, 4] *= 2.0 ** -100
    out = pisa.cache_attention(q, cache, i32([2999]))
    check_attention(cache, q, [2999], out)


def test_many_small_weights():
    """100000 keys of weight about 2^-20 of the largest: their part of the sum is not lost."""
    n = 100000
    cache = make_cache(gen(1), 1, n, 1, 64, 4, fill=False)
    k = torch.zeros(1, n, 1, 64, dtype=torch.bfloat16, device=DEV)
    v = torch.ones(1, n, 1, 64, dtype=torch.bfloat16, device=DEV)
    k[0, 5, 0, 0] = 6.0
    v[0, 5] = -1.0
    pisa.cache_append(None, k, v, cache, i32([0]), None)
    q = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = torch.linspace(15, 19, 16, device=DEV).to(torch.bfloat16)
    out = torch.empty(1, 1, 16, 64, dtype=torch.float32, device=DEV)
    pisa.cache_attention(q, cache, i32([n]), out=out)
    check_attention(cache, q, [n], out)


def test_offsets_past_32_bits():
    """Pages more than 4 GB apart."""
    for bits in (16, 4):
        inner = (1, 1, 2, 64, 64) if bits == 16 else (1, 1, 72 * 64)
        dt = torch.bfloat16 if bits == 16 else torch.uint8
        size = 2 if bits == 16 else 1
        step = (5 << 30) // size // 2
        pool = torch.zeros(2 * step + (1 << 20), dtype=dt, device=DEV)
        stride, strides = 1, []
        for s in reversed(inner):
            strides.insert(0, stride)
            stride *= s
        pages = torch.as_strided(pool, (3,) + inner, (step,) + tuple(strides))
        cache = pisa.PagedCache(pages, i32([[2, 0, 1]]), 64)
        g = gen(13)
        q, k, v = normal(g, 1, 150, 16, 64), normal(g, 1, 150, 1, 64), normal(g, 1, 150, 1, 64)
        _, ko = pisa.cache_append(None, k, v, cache, i32([0]), pisa.rotary_table(200))
        kr, vr = pisa.cache_read(cache, i32([0]), 150)
        if bits == 16:
            assert torch.equal(kr, ko) and torch.equal(vr, v)
        check_attention(cache, q[:, -1:], [150], pisa.cache_attention(q[:, -1:], cache, i32([150])))
        idx = i32([[[[1, 0, 2]]]])
        check_attention(cache, q[:, -1:], [150], pisa.cache_attention(q[:, -1:], cache, i32([150]), idx=idx), idx=idx)
        del pool, pages, cache
        torch.cuda.empty_cache()


# ------------------------------------------------------------------------------- streams, graphs, a whole decode


def test_another_stream_and_its_allocations():
    g = gen(14)
    cache = make_cache(g, 2, 5000, 2, 64, 4)
    q = normal(g, 2, 1, 32, 64)
    lengths = i32([5000, 4000])
    want = pisa.cache_attention(q, cache, lengths)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [pisa.cache_attention(q, cache, lengths, stream=side) for _ in range(20)]
    k, v = pisa.cache_read(cache, i32([0, 0]), 4000, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    k2, v2 = pisa.cache_read(cache, i32([0, 0]), 4000)
    assert torch.equal(k, k2) and torch.equal(v, v2)


def test_binding_refusals():
    g = gen(15)
    cache = make_cache(g, 2, 100, 2, 64, 4)
    q, k = normal(g, 2, 1, 32, 64), normal(g, 2, 1, 2, 64)
    n, rotary = i32([1, 1]), pisa.rotary_table(100)
    bad = [
        lambda: pisa.cache_attention(q[:1], cache, n),
        lambda: pisa.cache_attention(q.float(), cache, n),
        lambda: pisa.cache_attention(q.cpu(), cache, n),
        lambda: pisa.cache_attention(q, cache, n.long()),
        lambda: pisa.cache_attention(q, cache, n.cpu()),
        lambda: pisa.cache_attention(q, cache, n, idx=torch.zeros(2, 2, 2, 8, dtype=torch.int32, device=DEV)),
        lambda: pisa.cache_attention(q, cache, n, idx=torch.zeros(2, 2, 1, 0, dtype=torch.int32, device=DEV)),
        lambda: pisa.cache_attention(q, cache, n, out=q.half()),
        lambda: pisa.cache_append(q, k, k[:, :, :1], cache, n, rotary),
        lambda: pisa.cache_append(q, k, k, cache, n, rotary.double()),
        lambda: pisa.cache_append(q, k, k, cache, n, rotary[:, :40].contiguous()),
        lambda: pisa.cache_append(None, k, k, cache, n, rotary, q_out=q),
        lambda: pisa.cache_append(q, k, k, cache, n, rotary, k_out=k[:, :, :1].expand(2, 1, 2, 64)),
        lambda: pisa.cache_append(q.transpose(2, 3).contiguous().transpose(2, 3), k, k, cache, n, rotary),
        lambda: pisa.cache_read(cache, n, 0),
        lambda: pisa.cache_read(cache, n[:1], 1),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: pisa.cache_attention(normal(g, 2, 17, 32, 64), cache, n),
              lambda: pisa.cache_attention(normal(g, 2, 1, 6, 64), cache, n),
              lambda: pisa.cache_attention(q, cache, n, idx=torch.zeros(2, 2, 1, 65, dtype=torch.int32, device=DEV)),
              lambda: pisa.cache_attention(q, cache, n, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises(pisa.PisaError):
            f()


@pytest.mark.parametrize("bits", [16, 4])
def test_prefill_then_decode_steps_eager_and_captured(bits):
    """A prompt, then decode steps: append, select by the pyramid, attend over the selected blocks; the steps run
    eagerly and as replays of one captured graph give the same bits, and agree with 64 bits."""
    B, N, Hq, Hkv, K, steps, cap = 2, 700, 32, 2, 4, 5, 800
    g = gen(16)
    rotary = pisa.rotary_table(cap)

    def prompt():
        h = gen(17)
        cache = make_cache(h, B, cap, Hkv, 64, bits, fill=False)
        pyr = pisa.Pyramid.allocate(torch.zeros(B, cap, Hkv, 64, dtype=torch.bfloat16, device=DEV), with_lengths=True)
        q, k, v = normal(h, B, N, Hq, 64), normal(h, B, N, Hkv, 64), normal(h, B, N, Hkv, 64)
        q, _ = pisa.cache_append(q, k, v, cache, i32([0] * B), rotary, k_out=pyr.keys[:, :N])
        pisa.build_pyramid(pyr, N=N)
        idx, _ = pisa.select_prefill(q[:, :N], pyr, K, N=N, with_scores=False)
        return cache, pyr, q, idx

    cache, pyr, q, idx = prompt()
    # the prompt's last queries over their selected blocks
    T = 16
    last = pisa.cache_attention(q[:, N - T:], cache, i32([N] * B), idx=idx[:, :, N - T:].contiguous())
    check_attention(cache, q[:, N - T:], [N] * B, last, idx=idx[:, :, N - T:])
    new = [(normal(g, B, 1, Hq, 64), normal(g, B, 1, Hkv, 64), normal(g, B, 1, Hkv, 64)) for _ in range(steps)]
    ws, dws = pisa.cache_workspace(cache), torch.empty(pisa.decode_workspace_bytes(B, Hq, Hkv, K), dtype=torch.uint8, device=DEV)

    def step(cache, pyr, q, k, v, ws):
        qr, kr = pisa.cache_append(q, k, v, cache, pyr.lengths, rotary, workspace=ws)
        idx, _ = pisa.decode_append_and_select(qr.view(B, Hq, 64), kr.view(B, Hkv, 64), pyr, K, with_scores=False,
                                               workspace=dws)
        sel = pisa.cache_attention(qr, cache, pyr.lengths, idx=idx, workspace=ws)
        return qr, idx, sel, pisa.cache_attention(qr, cache, pyr.lengths, workspace=ws)

    eager = []
    for s in range(steps):
        qr, idx, sel, everything = step(cache, pyr, *new[s], ws)
        n = [N + s + 1] * B
        assert pyr.lengths.tolist() == n
        check_attention(cache, qr, n, sel, idx=idx[:, :, None])
        check_attention(cache, qr, n, everything)
        eager.append((idx.clone(), sel, everything))
    assert status(ws) == 0
    # the same from a fresh prompt, as replays of one graph
    cache2, pyr2, _, _ = prompt()
    q, k, v = (x.clone() for x in new[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # load every kernel before the capture, on a cache of its own
        step(*prompt()[:2], q, k, v, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(cache2, pyr2, q, k, v, ws)
    for s in range(steps):
        for dst, src in zip((q, k, v), new[s]):
            dst.copy_(src)
        graph.replay()
        for a, b in zip(got[1:], eager[s]):
            assert torch.equal(a, b), s
    assert torch.equal(cache.pages, cache2.pages) and status(ws) == 0


def test_two_graphs_with_one_workspace():
    """Two captured calls that share a workspace, replayed one after the other in any order."""
    g = gen(18)
    ws = None
    made = []
    for bits, lengths in ((16, [9000, 3000]), (4, [20000, 1])):
        cache = make_cache(g, 2, max(lengths), 2, 64, bits)
        ws = pisa.cache_workspace(cache) if ws is None else ws
        q, n = normal(g, 2, 1, 32, 64), i32(lengths)
        want = pisa.cache_attention(q, cache, n)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = pisa.cache_attention(q, cache, n, workspace=ws)
        made.append((graph, out, want, cache, q, n))
    for which in (0, 1, 1, 0, 0, 1, 0):
        made[which][1].zero_()
        made[which][0].replay()
        assert torch.equal(made[which][1], made[which][2])
    assert status(ws) == 0


@pytest.mark.parametrize("bits", [16, 4])
def test_many_sequences_in_a_long_table(bits):
    """257 sequences, many empty, in a table long enough that the tiles of all are one stream."""
    g = gen(19)
    B = 257
    cache = make_cache(g, 8, 2304, 2, 64, bits)
    lengths = [(b * 7919) % 2300 if b % 3 else 0 for b in range(B)]
    table = cache.table[torch.arange(B, device=DEV) % 8].contiguous()  # sequences share pages
    many = pisa.PagedCache(cache.pages, table, 64)
    q = normal(g, B, 2, 8, 64)
    ws = pisa.cache_workspace(many)
    out = torch.full((B, 2, 8, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    pisa.cache_attention(q, many, i32(lengths), out=out, workspace=ws)
    assert status(ws) == 0
    some = [b for b in range(B) if b % 16 == 1 or lengths[b] < 3]
    for b in some:
        one = pisa.PagedCache(cache.pages, table[b:b + 1].contiguous(), 64)
        check_attention(one, q[b:b + 1], lengths[b:b + 1], out[b:b + 1])
    o32 = torch.full((B, 2, 8, 64), 7.0, dtype=torch.float32, device=DEV)
    pisa.cache_attention(q, many, i32(lengths), out=o32, workspace=ws)
    for b in range(B):
        if lengths[b] == 0:
            assert bool((out[b] == 0).all()) and bool((o32[b] == 0).all())


@pytest.mark.parametrize("bits", [16, 4])
def test_calls_do_not_overtake_one_another(bits):
    """Kernels of later calls may start early, but the cache is not written while an earlier call reads it."""
    g = gen(20)
    tiles = 12  # no unit is cut: the joining kernel has nothing to wait for but the order
    n = tiles * (64 if bits == 4 else 32)
    cache = make_cache(g, 1, 4096, 2, 64, bits)
    start, lengths = i32([0]), i32([n])
    q = normal(g, 1, 1, 32, 64)
    new = [(normal(g, 1, n, 2, 64), normal(g, 1, n, 2, 64)) for _ in range(4)]
    ws = pisa.cache_workspace(cache)
    want = []
    for k, v in new:
        pisa.cache_append(None, k, v, cache, start, None)
        torch.cuda.synchronize()
        want.append(pisa.cache_attention(q, cache, lengths, workspace=ws).clone())
        torch.cuda.synchronize()
    outs, reads = [], []
    for i in range(40):
        k, v = new[i % 4]
        pisa.cache_append(None, k, v, cache, start, None, k_out=k)
        outs.append(pisa.cache_attention(q, cache, lengths, workspace=ws))
        reads.append(pisa.cache_read(cache, start, n))
    torch.cuda.synchronize()
    for i in range(40):
        assert torch.equal(outs[i], want[i % 4]), i
        assert torch.equal(reads[i][0], reads[i % 4][0]) and torch.equal(reads[i][1], reads[i % 4][1])


def in_a_wide_table(cache, tokens=20000):
    """The same cache with room for many more tokens, on pages that do not exist yet: the tiles of all
    sequences are then one stream, however short they are."""
    more = -(-tokens // cache.page_size)
    table = torch.cat([cache.table, torch.full((cache.B, more), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
    return pisa.PagedCache(cache.pages, table, cache.page_size, cache._struct.k_exp, cache._struct.v_exp)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("B,T,G,Hkv,page,lengths", ALL)
def test_attention_over_all_in_a_wide_table(bits, B, T, G, Hkv, page, lengths):
    g = gen(B * 100 + T + 1)
    cache = in_a_wide_table(make_cache(g, B, max(lengths) + 40, Hkv, page, bits, layers=2))
    q = normal(g, B, T, G * Hkv, 64)
    ws = pisa.cache_workspace(cache)
    out = torch.full((B, T, G * Hkv, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    pisa.cache_attention(q, cache, i32(lengths), out=out, workspace=ws)
    assert status(ws) == 0
    check_attention(cache, q, lengths, out)
    o32 = torch.full(out.shape, 7.0, dtype=torch.float32, device=DEV)
    pisa.cache_attention(q, cache, i32(lengths), out=o32, workspace=ws)
    check_attention(cache, q, lengths, o32)
    assert torch.equal(pisa.cache_attention(q, cache, i32(lengths), workspace=ws), out)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("T,G,page,n", [(1, 16, 64, 100), (4, 4, 16, 130), (3, 16, 128, 1665), (16, 1, 16, 2059)])
def test_what_a_query_does_not_see_in_a_wide_table(bits, T, G, page, n):
    g = gen(n + 1)
    cache = make_cache(g, 2, n + 150, 2, page, bits)
    q = normal(g, 2, T, 2 * G, 64)
    lengths = [n, n - 1]
    for b in range(2):
        for p in range(lengths[b], n + 64):
            poison(cache, b, p)
    cache.table[:, -(-n // page):] = -1
    cache = in_a_wide_table(cache)
    ws = pisa.cache_workspace(cache)
    check_attention(cache, q, lengths, pisa.cache_attention(q, cache, i32(lengths), workspace=ws))
    assert status(ws) == 0
    for what in ("k", "v"):
        for b in range(2):
            poison(cache, b, lengths[b] - 1, what)
        out = pisa.cache_attention(q, cache, i32(lengths))
        check_attention(cache, q, lengths, out, rows={(b, t) for b in range(2) for t in range(T - 1)})
        assert bool(torch.isnan(out[:, T - 1]).any(-1).all())


@pytest.mark.parametrize("bits", [16, 4])
def test_bad_pages_and_lengths_in_a_wide_table(bits):
    g = gen(21)
    short = make_cache(g, 3, 12000, 2, 64, bits)
    cache = in_a_wide_table(short, 64)
    q = normal(g, 3, 2, 16, 64)
    lengths = [12000, 11000, 130]
    cache.table[1, 100] = cache.n_pages  # in one of the several runs of its units
    ws = pisa.cache_workspace(cache)
    out = pisa.cache_attention(q, cache, i32(lengths), workspace=ws)
    assert status(ws) == 6
    assert bool(torch.isnan(out[1]).all())
    for b in (0, 2):
        good = pisa.PagedCache(cache.pages, cache.table[b:b + 1].contiguous(), 64)
        check_attention(good, q[b:b + 1], lengths[b:b + 1], out[b:b + 1])
    ws = pisa.cache_workspace(short)  # a length past the table's end is cut to it, and flagged
    full = short.max_pages * 64
    one = pisa.PagedCache(short.pages, short.table[:1].contiguous(), 64)
    long = pisa.cache_attention(q[:1], one, i32([full + 5]), workspace=ws)
    assert status(ws) == 6
    assert torch.equal(long, pisa.cache_attention(q[:1], one, i32([full])))


@pytest.mark.parametrize("bits", [16, 4])
def test_many_sequences_in_a_wide_table(bits):
    """257 sequences, many empty, some of them cut between runs."""
    g = gen(22)
    B = 257
    cache = make_cache(g, 8, 2304, 2, 64, bits)
    lengths = [(b * 7919) % 2300 if b % 3 else 0 for b in range(B)]
    table = cache.table[torch.arange(B, device=DEV) % 8].contiguous()
    many = in_a_wide_table(pisa.PagedCache(cache.pages, table, 64))
    q = normal(g, B, 2, 8, 64)
    ws = pisa.cache_workspace(many)
    out = torch.full((B, 2, 8, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    pisa.cache_attention(q, many, i32(lengths), out=out, workspace=ws)
    assert status(ws) == 0
    for b in [b for b in range(B) if b % 16 == 1 or lengths[b] < 3]:
        one = pisa.PagedCache(cache.pages, table[b:b + 1].contiguous(), 64)
        check_attention(one, q[b:b + 1], lengths[b:b + 1], out[b:b + 1])


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("B,T,G,Hkv,page,lengths", [
    (2, 3, 16, 2, 64, [9000, 777]),
    (1, 5, 16, 1, 32, [30011]),
    (3, 9, 16, 3, 16, [4097, 8, 10001]),
    (40, 4, 8, 1, 64, [9001] + [(37 * b) % 1900 for b in range(1, 40)]),
])
def test_several_row_tiles_over_runs(bits, B, T, G, Hkv, page, lengths):
    """Queries of 2 to 9 row tiles, which do not divide the grid, over units that lie in several runs."""
    g = gen(B * 100 + T + 2)
    cache = make_cache(g, B, max(lengths) + 40, Hkv, page, bits)
    q = normal(g, B, T, G * Hkv, 64)
    ws = pisa.cache_workspace(cache)
    out = torch.full((B, T, G * Hkv, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    pisa.cache_attention(q, cache, i32(lengths), out=out, workspace=ws)
    assert status(ws) == 0
    check_attention(cache, q, lengths, out)
    o32 = torch.full(out.shape, 7.0, dtype=torch.float32, device=DEV)
    pisa.cache_attention(q, cache, i32(lengths), out=o32, workspace=ws)
    check_attention(cache, q, lengths, o32)
    assert torch.equal(pisa.cache_attention(q, cache, i32(lengths), workspace=ws), out)


@pytest.mark.parametrize("n", [1, 100, 9000])
def test_rows_whose_logits_are_all_minus_infinity(n):
    """They get zeros, like rows that see nothing; the other rows of the tile are as ever."""
    g = gen(23)
    cache = make_cache(g, 1, n, 1, 64, 16)
    cache.pages[:, :, :, 0, :, 5] = float("-inf")
    q = normal(g, 1, 1, 16, 64)
    q[..., 5] = 0.5
    out = pisa.cache_attention(q, cache, i32([n]))
    assert bool((out == 0).all())
    one = int(cache.table[0, 0])
    cache.pages[one, 0, 0, 0, 0, 5] = 0.25  # token 0 is finite: it has all the weight
    out = pisa.cache_attention(q, cache, i32([n]))
    want = cache.pages[one, 0, 0, 1, 0]
    assert torch.equal(out[0, 0], want.expand(16, 64))


@pytest.mark.parametrize("B,T,Hq,Hkv,page,bits,rot", [
    (3, 1, 12, 3, 16, 16, 64), (2, 37, 5, 5, 64, 4, 64), (1, 1, 1, 1, 32, 4, 64), (2, 9, 40, 5, 128, 16, 64),
    (1, 2500, 8, 1, 64, 4, 64), (2, 30, 12, 3, 64, 16, 48), (2, 30, 20, 5, 16, 4, 32), (1, 31, 1, 1, 64, 16, 16),
])
def test_append_of_odd_head_counts(B, T, Hq, Hkv, page, bits, rot):
    """Query rows that do not fill their last group, in place and out of place."""
    g = gen(B * 1000 + T + rot)
    n_cap = T + 70
    cache = make_cache(g, B, n_cap, Hkv, page, bits, fill=False)
    before = cache.pages.clone()
    qkv = normal(g, B, T, Hq + 2 * Hkv, 64)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 2)
    start, counts = [5 * b for b in range(B)], [T if b == 0 else T // 2 for b in range(B)]
    rotary = pisa.rotary_table(n_cap, rot)
    ws = pisa.cache_workspace(cache)
    q_out = torch.full((B, T, Hq, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    k_out = torch.full((B, T, Hkv, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    pisa.cache_append(q, k, v, cache, i32(start), rotary, counts=i32(counts), q_out=q_out, k_out=k_out, workspace=ws)
    assert status(ws) == 0
    check_append(cache, q, k, v, start, counts, rotary, False, q_out, k_out, before)
    for b in range(B):
        assert bool((q_out[b, counts[b]:] == 7).all()) and bool((k_out[b, counts[b]:] == 7).all())
    whole = qkv.clone()
    qi, ki, vi = qkv.split([Hq, Hkv, Hkv], 2)
    pisa.cache_append(qi, ki, vi, cache, i32(start), rotary, counts=i32(counts), q_out=qi, k_out=ki, workspace=ws)
    for b in range(B):
        c = counts[b]
        assert torch.equal(qi[b, :c], q_out[b, :c]) and torch.equal(ki[b, :c], k_out[b, :c])
        assert torch.equal(qkv[b, c:], whole[b, c:]) and torch.equal(vi[b], whole[b, :, Hq + Hkv:])
