"""Lists that a pool's calls write may not lie in those that they still read: refused before any launch."""
import ctypes

import pytest

import pyramid_top_block_gb300 as pisa
from test_more_cache_abi import pool

B, MAX_PAGES, N_PAGES = 100, 4, 9
TABLE, REFS, LENGTHS, COUNTS = 0x20000, 0x30000, 0x40000, 0x48000
INSIDE = [0, 4, 4 * (B - 1), -4, -4 * (B - 1)]  # where a list of B entries begins that shares some with one at 0


def a_pool():
    return ctypes.byref(pool(B=B, max_pages=MAX_PAGES, n_pages=N_PAGES, table=TABLE, refs=REFS))


def reserve(granted, counts=COUNTS):
    lib = pisa.load()
    need = lib.pisa_pool_workspace_bytes(N_PAGES, B)
    return lib.pisa_cache_reserve(a_pool(), LENGTHS, 1, counts, granted, 0x60000, need, None)


@pytest.mark.parametrize("at", INSIDE)
def test_granted_in_lengths(at):
    """The lengths are read again after the first grants are written: pages would be looked up past the list."""
    assert reserve(LENGTHS + at) == 1 and reserve(LENGTHS + at, counts=None) == 1


@pytest.mark.parametrize("at", INSIDE[1:])
def test_granted_beside_counts(at):
    assert reserve(COUNTS + at) == 1


@pytest.mark.parametrize("granted", [TABLE, TABLE + 4 * (B * MAX_PAGES - 1), REFS + 4 * (N_PAGES - 1),
                                     REFS - 4 * (B - 1)])
def test_granted_in_the_pool(granted):
    assert reserve(granted) == 1


@pytest.mark.parametrize("at", INSIDE)
def test_parents_in_lengths(at):
    """Both are read by CTAs that may come after the lengths are written."""
    assert pisa.load().pisa_cache_fork(a_pool(), LENGTHS + at, LENGTHS, None, None) == 1


@pytest.mark.parametrize("x", [TABLE, TABLE + 4 * (B * MAX_PAGES - 1), REFS, REFS + 4 * (N_PAGES - 1)])
def test_lengths_and_used_in_the_pool(x):
    lib = pisa.load()
    need = lib.pisa_pool_workspace_bytes(N_PAGES, B)
    assert lib.pisa_cache_fork(a_pool(), 0x50000, x, None, None) == 1
    assert lib.pisa_cache_compact(a_pool(), x, 0x60000, need, None) == 1
