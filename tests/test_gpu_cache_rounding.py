"""The rotation where 32-bit sums do not decide the bf16 result: elements next to a border between two of them."""
import pytest
import torch

import cache_ref as ref
import pyramid_top_block_gb300 as pisa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rows_at_borders(n, H, rot, interleaved, seed):
    """bf16 rows [1, n, H, 64] and a table [n, rot] such that of every pair (a, b) one turned member lies, in most
    rows of head 0, within some 2^-24 of a value half way between two bf16; and the other heads as they come."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(1, n, H, 64, generator=g).to(torch.bfloat16)
    x = torch.where(x.abs() < 2.0 ** -6, torch.ones_like(x), x)
    i = torch.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[0, :, 0, ia].double(), x[0, :, 0, ib].double()  # [n, rot / 2]
    s = torch.rand(n, rot // 2, generator=g, dtype=torch.float64).float().double() * 2 - 1
    s = s.float().double()
    half = torch.randn(n, rot // 2, generator=g).to(torch.bfloat16).double()
    half = half + torch.ldexp(torch.ones_like(half), torch.frexp(half).exponent - 9)  # half of a bf16's step on
    # a c - b s, or b c + a s, next to the border
    c = torch.where(i % 2 == 0, (half + b * s) / a, (half - a * s) / b).float().double()
    return x, torch.cat([c, s], 1).float()


@pytest.mark.parametrize("rot,interleaved,Hq", [(64, False, 8), (64, False, 5), (64, True, 8), (32, False, 4),
                                               (48, True, 3)])
def test_rotation_at_the_borders(rot, interleaved, Hq):
    """Query and key rows (the kernel has a form of its own for each) get what the exact sum rounds to, by way of 32
    bits, whichever form turns them and in calls of any length."""
    n = 3000
    x, table = rows_at_borders(n, Hq, rot, interleaved, rot + Hq)
    x, table = x.to(DEV), table.to(DEV)
    pos = torch.arange(n, device=DEV)
    y = ref.rotate(x[0], table, pos, interleaved)  # 64 bits: off by 2^-53 of its products
    want = ref.to_bf16(y)
    # elements whose distance from a border between two fp32 values 64 bits, or the kernel's error term (2^-46 of the
    # products), cannot be sure of are left out
    mag = ref.rotate(x[0].abs(), torch.cat([table[:, :rot // 2].abs(), -table[:, rot // 2:].abs()], 1), pos,
                     interleaved).abs() + ref.rotate(x[0].abs(), table.abs(), pos, interleaved).abs()
    sure = ref.to_bf16(y - 2.0 ** -44 * mag) == ref.to_bf16(y + 2.0 ** -44 * mag)
    assert float(sure.double().mean()) > 0.99
    # the cases are what they are meant to be: 32-bit sums leave many elements of head 0 open
    open_ = ref.to_bf16(y - 2.0 ** -23 * mag) != ref.to_bf16(y + 2.0 ** -23 * mag)
    assert float(open_[:, 0].double().mean()) > 0.1
    U = 64
    pages = torch.zeros(-(-n // U), Hq, 1, 2, U, 64, dtype=torch.bfloat16, device=DEV)
    cache = pisa.PagedCache(pages, torch.arange(pages.shape[0], dtype=torch.int32, device=DEV)[None], U)
    start = torch.zeros(1, dtype=torch.int32, device=DEV)
    qo, ko = pisa.cache_append(x, x, x, cache, start, table, interleaved=interleaved)
    assert torch.equal(qo, ko)
    wrong = (qo[0] != want) & sure
    assert int(wrong.sum()) == 0, wrong.nonzero()[:5].tolist()
    for t in range(0, n, 61):  # a token by itself: many warps share it
        a, b = pisa.cache_append(x[:, t:t + 1], x[:, t:t + 1], x[:, t:t + 1], cache, start + t, table,
                                 interleaved=interleaved)
        assert torch.equal(a[0, 0], qo[0, t]) and torch.equal(b[0, 0], ko[0, t])
