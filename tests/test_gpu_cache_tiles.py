"""Every token of the cache counts once: equal weights over values that say where they come from."""
import pytest
import torch

import pyramid_top_block_gb300 as pisa
import test_gpu_cache as base

pytestmark = pytest.mark.gpu
DEV = base.DEV

# A token's value is 6 in one dim and zero elsewhere.  Which dim, in three codings: the first two name the token's
# tile of 32 among 4096 of them, the third its place in the tile (a tile lost and another read twice in its place
# differ in one of them).
CODINGS = {"tile": lambda p: p // 32 % 64, "stretch": lambda p: p // 2048 % 64, "token": lambda p: p % 64}


def fill(cache, coding, g, same_keys):
    """Values by the coding of their position, keys as they come or all the same; for every sequence of the table."""
    n = cache.max_pages * cache.page_size
    pos = torch.arange(n, device=DEV)
    v = torch.zeros(1, n, 1, 64, dtype=torch.bfloat16, device=DEV)
    v[0, pos, 0, CODINGS[coding](pos)] = 6.0
    v = v.expand(cache.B, n, cache.Hkv, 64)
    k = base.normal(g, 1, 1, cache.Hkv, 64) if same_keys else base.normal(g, 1, n, cache.Hkv, 64)
    pisa.cache_append(None, k.expand(cache.B, n, cache.Hkv, 64), v, cache,
                      torch.zeros(cache.B, dtype=torch.int32, device=DEV), None)


def check(cache, q, lengths, coding, seen_blocks=None):
    """Dim d is 6 times the share of the seen tokens whose code is d.

    The weights are equal (the same logit), 6 times their sum and their sum differ from those of exact numbers by
    the fp32 sums alone: a warp's sum over a run, the warps' and the runs' one after the other, fewer than 2^11
    additions deep for up to 131072 tokens (a lane adds a tile's 16 weights and the run's tiles after one another:
    131072 / 64 / 8 tiles at the most), 2^-24 each; and 2^-11 (fp16) or 2^-16 (bf16 parts) where a weight, which is a
    power of two or next to it, is rounded for the product with V.  In all less than 2^-10 of a share: less than one
    token in 1024, and no tile holds fewer than 32 of the 2048 tokens of its dim."""
    B, T, Hq, _ = q.shape
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
        ws = pisa.cache_workspace(cache)
        idx = None
        if seen_blocks is not None:
            idx = base.i32(seen_blocks).expand(B, cache.Hkv, T, len(seen_blocks)).contiguous()
        pisa.cache_attention(q, cache, base.i32(lengths), idx=idx, out=out, workspace=ws)
        assert base.status(ws) == 0
        for b, n in enumerate(lengths):
            for t in range(T):
                see = max(0, n - T + t + 1)
                pos = torch.arange(see, device=DEV)
                if seen_blocks is not None:
                    pos = pos[torch.isin(pos // 64, base.i32(seen_blocks).long())]
                count = torch.bincount(CODINGS[coding](pos), minlength=64).double()
                want = 6 * count / max(1, pos.numel())
                tol = want * (2.0 ** -10 + (torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else 0.0))
                err = (out[b, t].double() - want).abs()
                assert bool((err <= tol).all()), (b, t, coding, (err > tol).nonzero()[:4].tolist())


CASES = [
    # B, T, G, Hkv, page, lengths
    (1, 1, 16, 2, 64, [131071]),
    (1, 1, 16, 1, 16, [30011]),
    (1, 5, 16, 1, 32, [30011]),
    (2, 3, 16, 2, 64, [9000, 777]),
    (3, 9, 16, 3, 16, [4097, 8, 10001]),
    (2, 16, 4, 2, 128, [20017, 15]),
    (7, 1, 8, 2, 64, [12345, 0, 1, 64, 4096, 9999, 33]),
    (40, 4, 8, 1, 64, [9001] + [(37 * b) % 1900 for b in range(1, 40)]),
    (150, 1, 4, 2, 64, [(911 * b) % 5000 for b in range(150)]),
    (5, 3, 16, 2, 64, [1201, 2, 64, 66, 700]),
]


@pytest.mark.parametrize("coding", sorted(CODINGS))
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("B,T,G,Hkv,page,lengths", CASES)
def test_every_token_counts_once(bits, B, T, G, Hkv, page, lengths, coding):
    g = base.gen(B * 100 + T)
    cache = base.make_cache(g, B, max(lengths), Hkv, page, bits)
    # queries of zero over any keys; and any queries over keys that are all the same
    fill(cache, coding, g, same_keys=False)
    zero = torch.zeros(B, T, G * Hkv, 64, dtype=torch.bfloat16, device=DEV)
    check(cache, zero, lengths, coding)
    check(base.in_a_wide_table(cache), zero, lengths, coding)
    fill(cache, coding, g, same_keys=True)
    q = base.normal(g, B, T, G * Hkv, 64)
    check(cache, q, lengths, coding)
    check(base.in_a_wide_table(cache), q, lengths, coding)


@pytest.mark.parametrize("coding", ["tile", "token"])
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("B,T,G,Hkv,page,K,lengths", [(2, 1, 16, 2, 64, 64, [5000, 4097]), (1, 3, 4, 2, 16, 33, [4100]),
                                                     (90, 2, 8, 2, 32, 7, [(97 * b) % 1000 for b in range(90)])])
def test_every_listed_token_counts_once(bits, B, T, G, Hkv, page, K, lengths, coding):
    g = base.gen(B * 100 + K)
    cache = base.make_cache(g, B, max(lengths), Hkv, page, bits)
    fill(cache, coding, g, same_keys=True)
    blocks = torch.randperm(80, generator=torch.Generator().manual_seed(K))[:K].tolist()
    check(cache, base.normal(g, B, T, G * Hkv, 64), lengths, coding, blocks)


@pytest.mark.parametrize("k_exp,v_exp", [(-3, 5), (2, -24), (-24, 24), (1, 0)])
def test_exponents_of_the_cache(k_exp, v_exp):
    """Attention over 4-bit pages that hold keys and values divided by a power of two."""
    g = base.gen(40)
    for B, T, G, Hkv, page, lengths in ((2, 1, 16, 2, 64, [700, 65]), (2, 5, 4, 2, 16, [300, 3]), (1, 1, 8, 1, 64, [9000])):
        cache = base.make_cache(g, B, max(lengths) + 40, Hkv, page, 4, k_exp=k_exp, v_exp=v_exp)
        q = (base.normal(g, B, T, G * Hkv, 64) * 2.0 ** -k_exp).to(torch.bfloat16)
        for c in (cache, base.in_a_wide_table(cache)):
            for dtype in (torch.bfloat16, torch.float32):
                out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
                pisa.cache_attention(q, c, base.i32(lengths), out=out)
                base.check_attention(cache, q, lengths, out)
        idx = base.listed_blocks(g, B, Hkv, T, 5, lengths)
        base.check_attention(cache, q, lengths, pisa.cache_attention(q, cache, base.i32(lengths), idx=idx), idx=idx)


@pytest.mark.parametrize("B,T,Hq,Hkv,page,bits,rot", [
    (3, 1, 12, 3, 16, 16, 64), (2, 37, 5, 5, 64, 4, 64), (1, 1, 1, 1, 32, 4, 64), (2, 9, 40, 5, 128, 16, 64),
    (1, 2500, 8, 1, 64, 4, 64), (2, 30, 12, 3, 64, 16, 48), (2, 30, 20, 5, 16, 4, 32), (1, 31, 1, 1, 64, 16, 16),
])
def test_append_of_odd_head_counts_interleaved(B, T, Hq, Hkv, page, bits, rot):
    """Rows that do not fill their last group, pairs next to one another."""
    g = base.gen(B * 1000 + T + rot)
    cache = base.make_cache(g, B, T + 70, Hkv, page, bits, fill=False)
    before = cache.pages.clone()
    q, k, v = base.normal(g, B, T, Hq + 2 * Hkv, 64).split([Hq, Hkv, Hkv], 2)
    start, counts = [5 * b for b in range(B)], [T if b == 0 else T // 2 for b in range(B)]
    rotary = pisa.rotary_table(T + 70, rot)
    ws = pisa.cache_workspace(cache)
    q_out = torch.full((B, T, Hq, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    k_out = torch.full((B, T, Hkv, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    pisa.cache_append(q, k, v, cache, base.i32(start), rotary, counts=base.i32(counts), interleaved=True, q_out=q_out,
                      k_out=k_out, workspace=ws)
    assert base.status(ws) == 0
    base.check_append(cache, q, k, v, start, counts, rotary, True, q_out, k_out, before)
    for b in range(B):
        assert bool((q_out[b, counts[b]:] == 7).all()) and bool((k_out[b, counts[b]:] == 7).all())
