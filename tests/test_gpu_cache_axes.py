"""Rotation by positions on several axes, every output bit against 64 bits."""
import pytest
import torch

import cache_ref as ref
import pyramid_top_block_gb300 as pisa
from test_gpu_cache import DEV, check_append, gen, i32, make_cache, normal, status

pytestmark = pytest.mark.gpu


def row_of(rotary, positions, axes):
    """The cosines and sines that a token turns by, as a table's row [1, rot]."""
    half = rotary.shape[1] // 2
    at = torch.tensor([positions[a] for a in axes], device=rotary.device)
    i = torch.arange(half, device=rotary.device)
    return torch.cat([rotary[at, i], rotary[at, half + i]])[None]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("B,T,Hq,Hkv,page,rot,interleaved,axes", [
    (1, 1, 1, 1, 16, 16, False, [0] * 8),
    (3, 1, 32, 2, 64, 64, False, [0] * 8 + [1] * 12 + [2] * 12),
    (2, 7, 8, 1, 32, 64, True, [i % 3 for i in range(32)]),
    (1, 130, 32, 2, 64, 64, False, [i % 4 for i in range(32)]),
    (2, 33, 6, 3, 128, 48, False, [2] * 5 + [0] * 9 + [1] * 10),
    (1, 65, 4, 4, 256, 32, True, [3, 0, 1, 2] * 4),
])
def test_append_with_axes(bits, B, T, Hq, Hkv, page, rot, interleaved, axes):
    g = gen(B * 100 + T)
    cap, n_rot, A = T + 40, 500, max(axes) + 1
    cache = make_cache(g, B, cap, Hkv, page, bits, layers=2, k_exp=1 if bits == 4 else 0)
    q, k, v = normal(g, B, T, Hq + 2 * Hkv, 64).split([Hq, Hkv, Hkv], 2)
    rotary = pisa.rotary_table(n_rot, rot)
    start, counts = [(5 * b + 3) % 40 for b in range(B)], [max(1, T - 3 * b) for b in range(B)]
    positions = torch.randint(0, n_rot, (A, B, T), generator=g, device=DEV, dtype=torch.int32)
    positions[:, :, ::3] = positions[:1, :, ::3]  # text: all axes agree
    positions[:, 0, 0] = n_rot - 1
    before = cache.pages.clone()
    q_out, k_out = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    ws = pisa.cache_workspace(cache)
    pisa.cache_append(q, k, v, cache, i32(start), rotary, counts=i32(counts), interleaved=interleaved, q_out=q_out,
                      k_out=k_out, workspace=ws, positions=positions, axes=axes)
    assert status(ws) == 0
    # every token by a call's worth of plain rotation with a table of its own
    p = positions.tolist()
    for b in range(B):
        for t in range(counts[b]):
            row = row_of(rotary, [p[a][b][t] for a in range(A)], axes)
            zero = torch.tensor(0, device=DEV)
            assert torch.equal(q_out[b, t], ref.to_bf16(ref.rotate(q[b, t], row, zero, interleaved))), (b, t)
            assert torch.equal(k_out[b, t], ref.to_bf16(ref.rotate(k[b, t], row, zero, interleaved))), (b, t)
        assert bool((q_out[b, counts[b]:] == 7).all()) and bool((k_out[b, counts[b]:] == 7).all())
    # the pages hold the rotated keys and the values: as an append of them without rotation leaves them
    pages = cache.pages.clone()
    cache.pages.copy_(before)
    pisa.cache_append(None, k_out, v, cache, i32(start), None, counts=i32(counts))
    assert torch.equal(cache.pages, pages)


def test_axes_that_agree_are_the_plain_rotation():
    g = gen(3)
    for rot, interleaved in ((64, False), (64, True), (32, False)):
        cache = make_cache(g, 2, 200, 2, 64, 16)
        q, k, v = (normal(g, 2, 90, h, 64) for h in (32, 2, 2))
        rotary, start = pisa.rotary_table(300, rot), i32([100, 7])
        a = pisa.cache_append(q, k, v, cache, start, rotary, interleaved=interleaved)
        pages = cache.pages.clone()
        at = (start[:, None] + torch.arange(90, device=DEV)).to(torch.int32)
        b = pisa.cache_append(q, k, v, cache, start, rotary, interleaved=interleaved,
                              positions=at[None].repeat(3, 1, 1), axes=[i % 3 for i in range(rot // 2)])
        c = pisa.cache_append(q, k, v, cache, start, rotary, interleaved=interleaved, positions=at[None].contiguous())
        for x, y, z in zip(a, b, c):
            assert torch.equal(x, y) and torch.equal(x, z)
        assert torch.equal(pages, cache.pages)


def test_positions_out_of_range():
    """A token with a position outside the table on any axis is left out and flagged; the others are as ever."""
    g = gen(4)
    for T in (1, 12):
        cache = make_cache(g, 2, 40, 1, 16, 16)
        q, k, v = (normal(g, 2, T, h, 64) for h in (4, 1, 1))
        rotary, axes = pisa.rotary_table(50), [0] * 10 + [1] * 10 + [2] * 12
        positions = torch.randint(0, 50, (3, 2, T), generator=g, device=DEV, dtype=torch.int32)
        args = dict(positions=positions, axes=axes)
        qo, ko = pisa.cache_append(q, k, v, cache, i32([0, 3]), rotary, **args)
        for axis, value in ((0, -1), (1, 50), (2, 1 << 30)):
            bad = positions.clone()
            bad[axis, 1, T // 2] = value
            ws = pisa.cache_workspace(cache)
            q2, k2 = torch.full_like(qo, 7.0), torch.full_like(ko, 7.0)
            before = cache.pages.clone()
            pisa.cache_append(q, k, v, cache, i32([0, 3]), rotary, positions=bad, axes=axes, q_out=q2, k_out=k2, workspace=ws)
            assert status(ws) == 6
            keep = torch.ones(2, T, dtype=torch.bool, device=DEV)
            keep[1, T // 2] = False
            assert torch.equal(q2[keep], qo[keep]) and torch.equal(k2[keep], ko[keep])
            assert bool((q2[~keep] == 7).all()) and bool((k2[~keep] == 7).all()) and torch.equal(before, cache.pages)


def test_refusals():
    g = gen(5)
    cache = make_cache(g, 2, 40, 1, 16, 16)
    q, k, v = (normal(g, 2, 3, h, 64) for h in (4, 1, 1))
    rotary, start = pisa.rotary_table(50), i32([0, 3])
    p = torch.zeros(3, 2, 3, dtype=torch.int32, device=DEV)
    good = [0] * 16 + [2] * 16
    for kw in (dict(positions=p[0], axes=good), dict(positions=p.long(), axes=good), dict(positions=p[:, :1], axes=good),
               dict(positions=p, axes=good[:-1]), dict(positions=p, axes=good[:-1] + [3]), dict(positions=p, axes=good[:-1] + [-1]),
               dict(axes=good), dict(positions=p.cpu(), axes=good), dict(positions=p.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            pisa.cache_append(q, k, v, cache, start, rotary, **kw)
    with pytest.raises(ValueError):
        pisa.cache_append(q, k, v, cache, start, None, positions=p, axes=good)
    with pytest.raises(pisa.PisaError):
        pisa.cache_append(q, k, v, cache, start, rotary, positions=torch.zeros(5, 2, 3, dtype=torch.int32, device=DEV))
