"""The paged cache's operators in 64 bits, written out plainly (torch, any device)."""
import torch

D = 64
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
# every finite e4m3 value of sign + by its byte 0 .. 126
E4M3 = torch.tensor([(b & 7) * 2.0 ** -9 if b < 8 else (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10) for b in range(127)],
                    dtype=torch.float64)


def nearest(x, grid):
    """Index of the entry of an ascending grid nearest to x >= 0; halfway goes to the even index, past the end to
    the last."""
    grid = grid.to(x.device)
    hi = torch.searchsorted(grid, x.contiguous()).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    a, b = x - grid[lo], grid[hi] - x
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def quantise(x, exp=0):
    """x [..., 64] float64 -> (signed values / 2^exp / scale, scale bytes [..., 4])."""
    y = (x * 2.0 ** -exp).unflatten(-1, (4, 16))
    top = y.abs().amax(-1)
    s = nearest(torch.nan_to_num(top, nan=0.0, posinf=0.0) / 6, E4M3)
    scale = E4M3.to(x.device)[s][..., None]
    code = nearest(torch.nan_to_num(y.abs() / torch.where(scale > 0, scale, 1.0), nan=0.0, posinf=0.0), E2M1)
    v = E2M1.to(x.device)[code] * (scale > 0)
    bad = ~torch.isfinite(top)
    v = torch.where(bad[..., None], 0.0, torch.where(y < 0, -v, v))
    return v.flatten(-2), torch.where(bad, 127, s).to(torch.uint8)


def values(v, scales, exp=0):
    f = torch.cat([E4M3, torch.tensor([float("nan")], dtype=torch.float64)]).to(v.device)[scales.long()]
    return v * f.repeat_interleave(16, -1) * 2.0 ** exp


def unpack(codes):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = E2M1.to(codes.device)[c & 7]
    return torch.where(c >= 8, -v, v)


def tokens(cache, b, n):
    """K, V [n, Hkv, 64] float64 of a sequence's first n tokens."""
    U, P = min(cache.page_size, 64), cache.page_size
    pos = torch.arange(n, device=cache.pages.device)
    page = cache.table[b].long()[pos // P]
    rec, u = (pos % P) // U, pos % U
    kv = torch.arange(cache.Hkv, device=pos.device)
    r = cache.pages[page[:, None], kv, rec[:, None]]  # [n, Hkv, record]
    i = torch.arange(n, device=pos.device)
    if cache.bits == 16:
        return r[i, :, 0, u].double(), r[i, :, 1, u].double()
    out = []
    for k, exp in ((0, cache._struct.k_exp), (1, cache._struct.v_exp)):
        c = r[..., 36 * U * k:36 * U * k + 32 * U].unflatten(-1, (U, 32))[i, :, u]
        s = r[..., 36 * U * k + 32 * U:36 * U * (k + 1)].unflatten(-1, (U, 4))[i, :, u]
        out.append(values(unpack(c), s, exp))
    return tuple(out)


def rotate(x, table, pos, interleaved):
    """x [..., H, 64] (leading dims as pos) turned by rows pos of table; float64."""
    rot = table.shape[1]
    y = x.double().clone()
    c, s = table[pos].double()[..., None, :].chunk(2, -1)
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    xa, xb = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    return y


def to_bf16(x):
    """64 bits -> 32 -> bf16, as the rotation rounds."""
    return x.float().to(torch.bfloat16)


def attention(q, k, v, keep):
    """q [G, 64], k, v [n, 64] float64, keep int [n]: how often a key counts.  Returns (o, sum p |v|, sum |v|,
    largest sum |q k| / 8), zeros where no key counts."""
    z = q @ k.T / 8
    w = keep.double()
    seen = w > 0
    if not bool(seen.any()):
        return torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q), 0.0
    z = torch.where(seen, z, float("-inf"))
    p = torch.exp(z - z.amax(-1, keepdim=True)) * w
    p = torch.where(seen, p, 0.0)
    p = p / p.sum(-1, keepdim=True)
    big = float((q.abs() @ k[seen].abs().T / 8).max())
    a = v[seen].abs()
    return p[:, seen] @ v[seen], p[:, seen] @ a, (w[seen] @ a).expand_as(q), big


def tolerance(o, pv, sv, big, n, bits, out_dtype):
    """How far the kernel's o may be from 64 bits.  A weight is off, relative to itself, by
      2^-11 (fp16) or 2^-16 (two bf16 parts): its rounding for the product with V,
      2 * 2 * 64 * 2^-24 * big: the fp32 sum of 64 products in its logit and in the largest one (steps of up to
        2^-23 of the running sum, which `big` bounds), which the exponential turns into a relative error,
      2^-17: the exponential (2^-22) and the rounding of its argument (2^-24 of at most 64),
      n 2^-23: the fp32 sums over the keys;
    the weighted sum and the sum of the weights each, so twice, times sum p |v|; and the result's rounding.
    In fp16 a weight is held times 2^10, relative to a reference that is at most the largest weight, with steps of
    2^-24 at least (the subnormal numbers), so it is also off by up to half a step: 2^-25 / 2^10 = 2^-35 of the
    largest weight, which is at most 1.  That is 2^-35 times sum |v|, and what is left where the keys that carry the
    weight have a zero in some dim."""
    eps = (2.0 ** -11 if bits == 4 else 2.0 ** -16) + 256 * 2.0 ** -24 * big + 2.0 ** -17 + n * 2.0 ** -23
    pv = pv + (2.0 ** -35 / (2 * eps) * sv if bits == 4 else 0.0)
    return 2 * eps * pv + torch.finfo(out_dtype).eps / 2 * (o.abs() + 2 * eps * pv)
