"""Attention with capped scores, a bias by distance and a span of tokens for each query, in 64 bits, written out
plainly (torch, any device)."""
import torch


def attention(q, k, v, at, lo, hi, cap=0.0, slopes=None):
    """q [T, Hq, 64], k, v [n, Hkv, 64] float64; query t at position at[t] sees tokens lo[t] .. hi[t] - 1.  Returns
    (o, sum p |v|, largest sum |q k| / 8 of a seen token, largest |bias| of a token that counts), zeros for a query that
    sees nothing.  What a query does not see does not matter, whatever it holds."""
    T, Hq, _ = q.shape
    n, Hkv, _ = k.shape
    G = Hq // Hkv
    j = torch.arange(n, device=q.device)
    seen = (j >= lo[:, None]) & (j < hi[:, None])  # [T, n]
    o, pv = torch.zeros_like(q), torch.zeros_like(q)
    big = torch.zeros(T, Hq, 1, dtype=torch.float64, device=q.device)
    for h in range(Hq):
        x = q[:, h] @ k[:, h // G].T / 8
        x = torch.where(seen, x, 0.0)  # (a NaN that nobody sees)
        mag = torch.where(seen, torch.nan_to_num(q[:, h].abs() @ k[:, h // G].abs().T / 8, nan=0.0, posinf=0.0), 0.0)
        big[:, h] = mag.amax(1, keepdim=True)
        if cap:
            x = cap * torch.tanh(x / cap)
        if slopes is not None:
            x = x - float(slopes[h]) * (at[:, None] - j).abs()
        x = torch.where(seen, x, float("-inf"))
        top = x.amax(1, keepdim=True)
        p = torch.where(seen, torch.exp(x - torch.where(torch.isfinite(top), top, 0.0)), 0.0)
        s = p.sum(1, keepdim=True)
        p = torch.where(s > 0, p / s, 0.0)
        vis = v[:, h // G]
        if torch.isfinite(vis).all():
            o[:, h], pv[:, h] = p @ vis, p @ vis.abs()
        else:  # a value counts for those that see it alone
            clean = torch.nan_to_num(vis, nan=0.0, posinf=0.0, neginf=0.0)
            o[:, h], pv[:, h] = p @ clean, p @ clean.abs()
            for i in (~torch.isfinite(vis)).any(1).nonzero()[:, 0].tolist():
                odd = torch.where(torch.isfinite(vis[i]), 0.0, vis[i])
                o[:, h] += torch.where(seen[:, i, None], p[:, i, None] * odd, 0.0)
    return o, pv, big


def tolerance(o, pv, big, n, weight, out_dtype, cap=0.0):
    """How far the kernel's o may be from 64 bits.  A weight is off, relative to itself, by
      weight: its rounding for the product with V (2^-8: bf16, 2^-11: fp16, 2^-16: two bf16 parts),
      2 * 2 * 64 * 2^-24 * big: the fp32 sum of 64 products in its score and in the largest one (steps of up to 2^-23
        of the running sum, which `big` bounds), which the exponential turns into a relative error; a cap's slope is at
        most 1, so it makes none of this larger,
      2 * 16 * 2^-24 * min(big, cap): the cap's polynomial or exponentials, their products and the factors to base 2,
        16 roundings at most, of this score and of the largest one,
      2^-16: the exponential (2^-22) and the roundings of its argument and of the bias (2^-24 of at most 64 each, for
        weights above 2^-64 of the largest one; smaller ones are less than the rest of this),
      n 2^-23: the fp32 sums over the keys;
    the weighted sum and the sum of the weights each, so twice, times sum p |v|; and the result's rounding."""
    eps = weight + 256 * 2.0 ** -24 * big + 2.0 ** -16 + n * 2.0 ** -23
    if cap:
        eps = eps + 32 * 2.0 ** -24 * big.clamp(max=cap)
    return 2 * eps * pv + torch.finfo(out_dtype).eps / 2 * (o.abs() + 2 * eps * pv) + 2.0 ** -120
