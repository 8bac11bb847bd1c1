"""Argument checks of the scored, prompt, axes and pool entry points: everything here returns before any launch."""
import ctypes

import pytest
import torch

import pyramid_top_block_gb300 as pisa
from test_cache_abi import BAD_CACHE, cache, rows

NAN = float("nan")


def axes(c, n_axes=3, axis_of=0, positions=0x80000, rot=64, n_rot=100, T=1, rotary=0x50000):
    return pisa.load().pisa_cache_append_axes(ctypes.byref(c), T, rows(), 32, rows(), rows(), 0x40000, None, rotary, n_rot,
                                              rot, 0, positions, n_axes, axis_of, rows(), rows(), None, None)


def scored(c, cap=1.0, slopes=None, window=0, T=1, ws_bytes=None, idx=None, Ksel=0):
    need = pisa.cache_workspace_bytes() if ws_bytes is None else ws_bytes
    return pisa.load().pisa_cache_attention_scored(ctypes.byref(c), rows(), T, 32, 0x40000, idx, Ksel, cap, slopes, window,
                                                   0x50000, 0, 0x60000, need, None)


def prompt(c, q=rows(), T=40, Hq=32, start=0x40000, counts=None, first=None, last=None, cap=0.0, slopes=None, window=0,
           out=0x50000, ws=0x60000, ws_bytes=None):
    need = pisa.cache_workspace_bytes() if ws_bytes is None else ws_bytes
    return pisa.load().pisa_cache_prompt_attention(ctypes.byref(c), q, T, Hq, start, counts, first, last, cap, slopes,
                                                   window, out, ws, need, None)


@pytest.mark.parametrize("change,status", BAD_CACHE)
def test_bad_descriptors(change, status):
    c = cache(**change)
    assert axes(c) == status and scored(c) == status and prompt(c) == status


@pytest.mark.parametrize("change,status", [
    (dict(positions=None), 1), (dict(positions=0x80002), 1), (dict(n_axes=0), 1), (dict(n_axes=5), 2), (dict(rot=0), 1),
    (dict(rot=20), 2), (dict(rot=80), 2), (dict(axis_of=3), 1), (dict(axis_of=3 << 62), 1), (dict(n_axes=1, axis_of=1 << 20), 1),
    (dict(n_rot=(1 << 27) + 1), 2), (dict(n_rot=0), 1), (dict(rotary=None), 1), (dict(T=0), 1),
])
def test_axes_refusals(change, status):
    assert axes(cache(), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(cap=-1.0), 1), (dict(cap=NAN), 1), (dict(cap=1e-9), 2), (dict(cap=1e9), 2), (dict(cap=float("inf")), 2),
    (dict(window=-1), 1), (dict(slopes=0x70001), 1), (dict(T=17), 2), (dict(ws_bytes=512), 3),
    (dict(idx=0x70000, Ksel=65), 2),
])
def test_scored_refusals(change, status):
    assert scored(cache(), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=0), 1), (dict(Hq=0), 1), (dict(Hq=3), 2), (dict(Hq=64), 2), (dict(q=None), 1), (dict(start=None), 1),
    (dict(out=None), 1), (dict(ws=None), 1), (dict(ws=0x60010), 1), (dict(out=0x50008), 1), (dict(first=0x40002), 1),
    (dict(last=0x40001), 1), (dict(counts=0x40002), 1), (dict(cap=-2.0), 1), (dict(cap=1e30), 2), (dict(window=-5), 1),
    (dict(ws_bytes=4096), 3), (dict(T=(1 << 27) + 1), 2), (dict(T=1 << 29), 2),
])
def test_prompt_refusals(change, status):
    assert prompt(cache(), **change) == status


def pool(**kw):
    a = dict(pages=0x10000, table=0x20000, refs=0x30000, page_stride=1024, page_bytes=512, B=3, page_size=64, n_pages=9,
             max_pages=4)
    a.update(kw)
    return pisa._PoolStruct(*a.values())


BAD_POOL = [
    (dict(pages=None), 1), (dict(table=None), 1), (dict(refs=None), 1), (dict(pages=0x10008), 1), (dict(table=0x20002), 1),
    (dict(refs=0x30001), 1), (dict(page_stride=496), 1), (dict(page_stride=1032), 1), (dict(page_bytes=0), 1),
    (dict(page_bytes=500), 1), (dict(page_stride=1 << 62), 1), (dict(B=0), 1), (dict(B=65536), 2), (dict(page_size=0), 1),
    (dict(page_size=48), 2), (dict(n_pages=0), 1), (dict(n_pages=(1 << 30) + 1), 2), (dict(max_pages=0), 1),
    (dict(max_pages=(1 << 21) + 1), 2),
]


@pytest.mark.parametrize("change,status", BAD_POOL)
def test_bad_pools(change, status):
    lib, p = pisa.load(), ctypes.byref(pool(**change))
    assert lib.pisa_cache_fork(p, 0x40000, 0x50000, None, None) == status
    assert lib.pisa_cache_reserve(p, 0x40000, 1, None, 0x50000, 0x60000, 1 << 40, None) == status
    assert lib.pisa_cache_compact(p, 0x40000, 0x60000, 1 << 40, None) == status


def test_pool_refusals():
    lib, p = pisa.load(), ctypes.byref(pool())
    need = lib.pisa_pool_workspace_bytes(9, 3)
    assert need >= 256 + 4 * (64 + 27 + 9) and need % 256 == 0
    assert lib.pisa_pool_workspace_bytes(0, 3) == lib.pisa_pool_workspace_bytes(9, 0) == 0
    assert lib.pisa_cache_fork(p, None, 0x50000, None, None) == 1
    assert lib.pisa_cache_fork(p, 0x40000, None, None, None) == 1
    assert lib.pisa_cache_fork(p, 0x40000, 0x50002, None, None) == 1
    assert lib.pisa_cache_fork(ctypes.byref(pool(B=32769)), 0x40000, 0x50000, None, None) == 2
    ok = [p, 0x40000, 1, None, 0x50000, 0x60000, need, None]
    for at, value, status in ((1, None, 1), (1, 0x40001, 1), (2, 0, 1), (3, 0x40002, 1), (4, None, 1), (5, None, 1),
                              (5, 0x60010, 1), (6, need - 1, 3)):
        args = list(ok)
        args[at] = value
        assert lib.pisa_cache_reserve(*args) == status, (at, value)
    for args, status in (((p, None, 0x60000, need, None), 1), ((p, 0x40000, None, need, None), 1),
                         ((p, 0x40000, 0x60000, need - 1, None), 3), ((p, 0x40002, 0x60000, need, None), 1)):
        assert lib.pisa_cache_compact(*args) == status


def test_binding_refuses_host_pools():
    table, refs = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pisa.PagePool(torch.zeros(2, 16), table, refs, 64)
    with pytest.raises(ValueError, match="page_size"):
        pisa.PagePool(torch.zeros(2, 16), table, refs, 65)
    with pytest.raises(ValueError, match="16 bytes"):
        pisa.PagePool(torch.zeros(2, 3), table, refs, 64)
    with pytest.raises(ValueError):
        pisa.PagePool.allocate(1, 10, 1, 0, device="cpu")
