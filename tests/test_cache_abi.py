"""Argument checks of the paged cache's entry points: everything here returns before any launch."""
import ctypes

import pytest
import torch

import pyramid_top_block_gb300 as pisa

vp = ctypes.c_void_p
OK_STRIDES = (64 * 32, 64 * 32, 64)


def cache(**kw):
    a = dict(pages=0x10000, table=0x20000, page_stride=72 * 64 * 2, B=2, Hkv=2, d=64, page_size=64, n_pages=9,
             max_pages=4, kind=1, k_exp=0, v_exp=0)
    a.update(kw)
    return pisa._CacheStruct(*a.values())


def rows(data=0x30000, strides=OK_STRIDES):
    return ctypes.byref(pisa._RowsStruct(data, *strides))


BAD_CACHE = [
    (dict(pages=None), 1), (dict(table=None), 1), (dict(pages=0x10008), 1), (dict(table=0x20002), 1),
    (dict(B=0), 1), (dict(Hkv=0), 1), (dict(n_pages=0), 1), (dict(max_pages=0), 1), (dict(page_size=0), 1),
    (dict(page_size=48), 2), (dict(page_size=512), 2), (dict(page_size=8), 2), (dict(d=128), 2), (dict(Hkv=33), 2),
    (dict(B=40000), 2), (dict(kind=2), 2), (dict(max_pages=(1 << 21) + 1), 2), (dict(k_exp=25), 2),
    (dict(v_exp=-25), 2), (dict(kind=0, page_stride=256 * 64 * 2, k_exp=1), 2), (dict(page_stride=72 * 64 * 2 - 16), 1),
    (dict(page_stride=72 * 64 * 2 + 8), 1), (dict(page_stride=1 << 62), 1), (dict(kind=0), 1),
]


def append(c, T=1, q=rows(), Hq=32, k=rows(), v=rows(), start=0x40000, counts=None, rotary=0x50000, n_rot=100, rot=64,
           q_out=rows(), k_out=rows(), ws=None):
    return pisa.load().pisa_cache_append(ctypes.byref(c), T, q, Hq, k, v, start, counts, rotary, n_rot, rot, 0, q_out,
                                         k_out, ws, None)


def read(c, T=1, start=0x40000, counts=None, k_out=rows(), v_out=rows(), ws=None):
    return pisa.load().pisa_cache_read(ctypes.byref(c), T, start, counts, k_out, v_out, ws, None)


def attend(c, q=rows(), T=1, Hq=32, lengths=0x40000, idx=None, Ksel=0, out=0x50000, ws=0x60000, ws_bytes=None):
    need = pisa.cache_workspace_bytes() if ws_bytes is None else ws_bytes
    return pisa.load().pisa_cache_attention(ctypes.byref(c), q, T, Hq, lengths, idx, Ksel, out, 0, ws, need, None)


@pytest.mark.parametrize("change,status", BAD_CACHE)
def test_bad_descriptors(change, status):
    c = cache(**change)
    assert append(c) == status
    assert read(c) == status
    assert attend(c) == status


def test_null_descriptor():
    lib = pisa.load()
    assert lib.pisa_cache_read(None, 1, 0x40000, None, rows(), rows(), None, None) == 1


@pytest.mark.parametrize("change,status", [
    (dict(T=0), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(k=rows(0)), 1), (dict(start=None), 1),
    (dict(start=0x40002), 1), (dict(counts=0x40002), 1), (dict(ws=0x40002), 1), (dict(q_out=None), 1),
    (dict(k=rows(0x30008)), 1), (dict(q=rows(strides=(2048, 2048, 68))), 1), (dict(k_out=rows(strides=(4, 64, 64))), 1),
    (dict(rot=8), 2), (dict(rot=80), 2), (dict(rot=-16), 2), (dict(rotary=None), 1), (dict(rotary=0x50008), 1),
    (dict(n_rot=0), 1), (dict(Hq=0), 1), (dict(Hq=3), 2), (dict(Hq=64), 2), (dict(Hq=6), 2), (dict(T=1 << 30), 2),
])
def test_append_refusals(change, status):
    assert append(cache(), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=0), 1), (dict(start=None), 1), (dict(k_out=None, v_out=None), 1), (dict(k_out=rows(0x30004)), 1),
    (dict(T=(1 << 31) - 1), 2),
])
def test_read_refusals(change, status):
    assert read(cache(), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=0), 1), (dict(T=17), 2), (dict(q=None), 1), (dict(lengths=None), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(ws=0x60010), 1), (dict(out=0x50008), 1), (dict(idx=0x70002, Ksel=8), 1), (dict(idx=0x70000, Ksel=0), 2),
    (dict(idx=0x70000, Ksel=65), 2), (dict(Hq=0), 1), (dict(Hq=3), 2), (dict(Hq=64), 2), (dict(ws_bytes=1000), 3),
])
def test_attention_refusals(change, status):
    assert attend(cache(), **change) == status


def test_page_bytes():
    lib = pisa.load()
    assert lib.pisa_cache_page_bytes(64, 2, 0) == 64 * 2 * 256
    assert lib.pisa_cache_page_bytes(16, 8, 1) == 16 * 8 * 72
    for bad in ((20, 2, 0), (64, 0, 0), (64, 33, 0), (64, 2, 3)):
        assert lib.pisa_cache_page_bytes(*bad) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    table = torch.zeros(1, 2, dtype=torch.int32)
    good = torch.zeros(2, 1, 1, 2, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pisa.PagedCache(good, table, 64)
    with pytest.raises(ValueError, match="page_size"):
        pisa.PagedCache(good, table, 60)
    with pytest.raises(ValueError):
        pisa.PagedCache(good, table, 32)
    with pytest.raises(ValueError):
        pisa.PagedCache(good.float(), table, 64)
    with pytest.raises(ValueError, match="contiguous"):
        pisa.PagedCache(good.transpose(3, 4).contiguous().transpose(3, 4), table, 64)
    with pytest.raises(ValueError, match="table"):
        pisa.PagedCache(good, table.long(), 64)
    with pytest.raises(ValueError):
        pisa.rotary_table(10, rot=24, device="cpu")


def test_rotary_table():
    t = pisa.rotary_table(5, rot=16, base=100.0, device="cpu")
    assert t.shape == (5, 16) and t.dtype == torch.float32
    import math
    for p in range(5):
        for i in range(8):
            a = p * 100.0 ** (-2 * i / 16)
            assert abs(float(t[p, i]) - math.cos(a)) <= 2.0 ** -24 and abs(float(t[p, 8 + i]) - math.sin(a)) <= 2.0 ** -24
