"""What the paged cache's operators cost: cases, their inputs, plain forms, and the framework's own calls.

Three operators of one decoding path:

* ``append``: rotate the new queries and keys by their positions and put keys and values into a paged cache,
  whose pages hold bf16 or 4-bit values;
* ``attend``: the newest T tokens of each sequence attend over the paged cache, all of it or the key blocks
  (64 tokens) that a selection chose;
* ``read``: cached tokens back as dense bf16.

``own`` false: elementary torch operations in 32 bits (64 where a value next to a rounding border matters);
``own`` true: the framework's calls.

A page holds ``page`` tokens of every KV head as records of U = min(page, 64) tokens.  A bf16 record is
[2 (K, V), U, 64]; a 4-bit record is U x 72 bytes: K codes [U, 32], K scales [U, 4], V codes [U, 32], V scales
[U, 4].  A code byte holds dims 2i (low nibble) and 2i + 1 as e2m1; a scale byte is the e4m3 factor of 16 dims.
"""
import math
import random

import torch

own = False

D = 64
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # of the e2m1 codes 0..7; bit 3 is the sign
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one decoding step's rotation and cache write for a batch of long contexts (decode benchmark: 16 x 131072)
        dict(name="append step 16 4-bit", op="append", kind="e2m1", B=16, T=1, n=131072, Hq=32, Hkv=2, page=64,
             rot=64, interleaved=False, ragged=False),
        # one step of a larger batch of short contexts, four query heads per KV head, small pages
        dict(name="append step 65 bf16", op="append", kind="bf16", B=65, T=1, n=2049, Hq=16, Hkv=4, page=16,
             rot=64, interleaved=True, ragged=True),
        # a whole prompt of the latency benchmark's 32K size
        dict(name="append prompt 32768 bf16", op="append", kind="bf16", B=1, T=32768, n=32768, Hq=32, Hkv=2,
             page=64, rot=64, interleaved=False, ragged=False),
        # two ragged prompts (the ragged benchmark's size), rotation of half the dims
        dict(name="append prompts 2x16421 4-bit", op="append", kind="e2m1", B=2, T=16421, n=16421, Hq=32, Hkv=2,
             page=128, rot=32, interleaved=False, ragged=True),
        # the attention after a decode selection: 8 blocks per sequence and KV head out of 131072 tokens
        dict(name="attend 8 blocks 16x131072 4-bit", op="attend", kind="e2m1", B=16, T=1, n=131072, Hq=32, Hkv=2,
             page=64, K=8, ragged=False, out="bf16"),
        # the same over bf16 pages
        dict(name="attend 8 blocks 16x131072 bf16", op="attend", kind="bf16", B=16, T=1, n=131072, Hq=32, Hkv=2,
             page=64, K=8, ragged=False, out="bf16"),
        # a large batch with 32 blocks each, small pages, ragged contexts
        dict(name="attend 32 blocks 128x16421 4-bit", op="attend", kind="e2m1", B=128, T=1, n=16421, Hq=32, Hkv=2,
             page=16, K=32, ragged=True, out="bf16"),
        # a layer without selection: every cached token, long contexts
        dict(name="attend all 16x131072 4-bit", op="attend", kind="e2m1", B=16, T=1, n=131072, Hq=32, Hkv=2,
             page=64, K=0, ragged=False, out="bf16"),
        # the same over bf16 pages, ragged contexts
        dict(name="attend all 8x131072 bf16", op="attend", kind="bf16", B=8, T=1, n=131072, Hq=32, Hkv=2, page=64,
             K=0, ragged=True, out="bf16"),
        # a few speculative tokens over short ragged contexts, four query heads per KV head
        dict(name="attend all 5x1201 T=3 4-bit", op="attend", kind="e2m1", B=5, T=3, n=1201, Hq=8, Hkv=2, page=32,
             K=0, ragged=True, out="bf16"),
        # a swapped-in context's keys and values for a new pyramid
        dict(name="read 131072 4-bit", op="read", kind="e2m1", B=1, T=131072, n=131072, Hkv=2, page=64,
             ragged=False),
        # the newest tokens of short ragged contexts
        dict(name="read 7x300 bf16", op="read", kind="bf16", B=7, T=300, n=4096, Hkv=4, page=16, ragged=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "read"])
    c = dict(op=op, kind=rng.choice(["bf16", "e2m1"]), page=rng.choice([16, 32, 64, 128, 256]),
             Hkv=rng.choice([1, 2, 4, 8]), ragged=rng.random() < 0.6)
    G = rng.choice([1, 2, 4, 8, 16])
    if op == "append":
        c.update(B=_spread(rng, 1, 128), Hq=G * c["Hkv"])
        most = 900000 // (c["B"] * (c["Hq"] + 4 * c["Hkv"] + 8))
        c["T"] = 1 if rng.random() < 0.4 else _spread(rng, 2, max(2, min(most, 32768)))
        c.update(n=c["T"] + _spread(rng, 1, 131072 // c["B"]), rot=rng.choice([16, 32, 48, 64, 64]),
                 interleaved=rng.random() < 0.5)
    elif op == "read":
        c["B"] = _spread(rng, 1, 64)
        c["T"] = _spread(rng, 1, 262144 // (c["B"] * c["Hkv"]))
        c["n"] = c["T"] + _spread(rng, 1, 131072 // c["B"])
    else:
        c["B"] = _spread(rng, 1, 128)
        c["T"] = 1 if rng.random() < 0.6 else rng.randint(2, 16)
        rows = c["B"] * c["Hkv"] * c["T"]
        most = (1 << 22) // rows if c["kind"] == "e2m1" else (1 << 20) // rows
        c["K"] = 0 if rng.random() < 0.5 else min(_spread(rng, 1, 32), max(1, 16384 // rows))
        c["n"] = max(c["T"], _spread(rng, 1, max(1, min(262144, most))))
        c.update(Hq=G * c["Hkv"], out=rng.choice(["bf16", "bf16", "fp32"]) if c["kind"] == "bf16" else "bf16")
    return c


def lengths_of(c):
    """Tokens of each sequence after the case's call: n, or between 1 and n where the case is ragged."""
    if not c["ragged"]:
        return [c["n"]] * c["B"]
    r = random.Random(1000003 * c["B"] + c["n"])
    return [c["n"] if b == 0 else max(1, int(c["n"] * r.uniform(0.05, 1.0))) for b in range(c["B"])]


def counts_of(c):
    """Tokens of each sequence that an append or a read is about: at most T, and no more than there are."""
    return [min(c["T"], n) for n in lengths_of(c)]


def row_bytes(c):
    """Bytes of one token's keys and values of one KV head."""
    return 256 if c["kind"] == "bf16" else 72


def work(c):
    ns, per = lengths_of(c), row_bytes(c)
    if c["op"] == "append":
        tok = sum(counts_of(c))
        heads = c["Hq"] + c["Hkv"]
        # queries, keys and values in; rotated queries and keys and the pages out; one table row a token
        moved = tok * ((2 * heads + c["Hkv"]) * 2 * D + c["Hkv"] * per + 4 * c["rot"])
        if c["kind"] == "e2m1":  # and the values that the new codes stand for
            moved += tok * c["Hkv"] * (per + 4 * D)
        return dict(bytes=moved, flops=3 * c["rot"] * heads * tok)
    if c["op"] == "read":
        return dict(bytes=sum(counts_of(c)) * c["Hkv"] * (per + 4 * D), flops=0)
    G, T = c["Hq"] // c["Hkv"], c["T"]
    outs = c["B"] * T * c["Hq"] * D * (2 + (2 if c["out"] == "bf16" else 4))
    if not c["K"]:
        seen = sum(max(0, n - T + t + 1) for n in ns for t in range(T)) * c["Hkv"]
        return dict(bytes=sum(ns) * c["Hkv"] * per + outs, flops=4 * D * G * seen)
    blocks = sum(min(c["K"], -(-(n - T + t + 1) // 64)) for n in ns for t in range(T) if n - T + t >= 0) * c["Hkv"]
    return dict(bytes=blocks * (64 * per + 4) + outs, flops=4 * D * G * 64 * blocks)


def quantised(x):
    """float [..., 64] -> (codes uint8 [..., 32], scales uint8 [..., 4]): one e4m3 scale per 16 values, the largest
    of them at 6; nearest code, a value half way between two to the even code, past the largest the largest."""
    y = x.unflatten(-1, (4, 16))
    scale = (y.abs().amax(-1).double() / 6).clamp(max=448.0).float().to(E4M3)
    s = scale.float().unsqueeze(-1)
    r = y.abs().double() / torch.where(s > 0, s, 1.0).double()
    code = torch.zeros(r.shape, dtype=torch.uint8, device=x.device)
    for i in range(7):  # the border between codes i and i + 1 goes to the even one
        border = (MAGNITUDES[i] + MAGNITUDES[i + 1]) / 2
        code += (r >= border) if i % 2 else (r > border)
    code = torch.where(s > 0, code, 0) | (torch.signbit(y).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def dequantised(codes, scales):
    """The values of codes uint8 [..., 32] and scales uint8 [..., 4]: fp32 [..., 64]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    return (table[c].unflatten(-1, (4, 16)) * scales.view(E4M3).float().unsqueeze(-1)).flatten(-2)


def views(s):
    """The pages as (K, V) of bf16 [n_pages, Hkv, records, U, 64], or as (K codes, K scales, V codes, V scales)."""
    U = min(s["page"], 64)
    if s["kind"] == "bf16":
        return s["pages"][:, :, :, 0], s["pages"][:, :, :, 1]
    p = s["pages"]
    return (p[..., :32 * U].unflatten(-1, (U, 32)), p[..., 32 * U:36 * U].unflatten(-1, (U, 4)),
            p[..., 36 * U:68 * U].unflatten(-1, (U, 32)), p[..., 68 * U:].unflatten(-1, (U, 4)))


def places(s, b, pos):
    """(page, record, row) of position pos of sequence b (tensors that broadcast together)."""
    U = min(s["page"], 64)
    page = s["table"][b, pos // s["page"]].long()
    return page, (pos % s["page"]) // U, pos % U


def prepare(case, seed):
    c = dict(case)
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(torch.bfloat16)

    B, T, n, Hkv, P = c["B"], c["T"], c["n"], c["Hkv"], c["page"]
    U = min(P, 64)
    per = -(-n // P)  # pages of a sequence
    n_pages = B * per + 3  # a pool with pages that no sequence holds
    s = dict(c, table=torch.randperm(n_pages, generator=g, device=dev)[:B * per].view(B, per).to(torch.int32))
    ns = torch.tensor(lengths_of(c), dtype=torch.int32, device=dev)
    s["lengths"] = ns
    # keys with a scale of their own per dim, as projections have them, values around one
    k_scale = torch.rand(D, generator=g, device=dev) * 1.5 + 0.25
    if c["kind"] == "bf16":
        s["pages"] = torch.empty(n_pages, Hkv, P // U, 2, U, D, dtype=torch.bfloat16, device=dev)
        kp, vp = views(s)
        kp.copy_(torch.randn(kp.shape, generator=g, device=dev, dtype=torch.float32) * k_scale)
        vp.copy_(torch.randn(vp.shape, generator=g, device=dev, dtype=torch.float32))
    else:
        s["pages"] = torch.empty(n_pages, Hkv, P // U, U * 72, dtype=torch.uint8, device=dev)
        kc, ks, vc, vs = views(s)
        chunk = max(1, (1 << 25) // (Hkv * P * D))
        for i in range(0, n_pages, chunk):
            shape = kc[i:i + chunk].shape[:-1] + (D,)
            for codes, scales, amp in ((kc, ks, k_scale), (vc, vs, 1.0)):
                x = (torch.randn(shape, generator=g, device=dev) * amp).to(torch.bfloat16).float()
                codes[i:i + chunk], scales[i:i + chunk] = quantised(x)
    if c["op"] != "attend":
        s["counts"] = torch.tensor(counts_of(c), dtype=torch.int32, device=dev)
        s["start"] = ns - s["counts"]
        s["k_out"] = torch.zeros(B, T, Hkv, D, dtype=torch.bfloat16, device=dev)
    if c["op"] == "append":
        # the three projections of one fused product, side by side in a token's row
        qkv = normal(B, T, c["Hq"] + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv.split([c["Hq"], Hkv, Hkv], dim=2)
        s["k"] *= k_scale.to(torch.bfloat16)
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
        angle = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * inv
        s["rotary"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["q_out"] = torch.zeros(B, T, c["Hq"], D, dtype=torch.bfloat16, device=dev)
    if c["op"] == "read" or (c["op"] == "append" and c["kind"] == "e2m1"):
        s["k_read"] = torch.zeros(B, T, Hkv, D, dtype=torch.bfloat16, device=dev)
        s["v_read"] = torch.zeros(B, T, Hkv, D, dtype=torch.bfloat16, device=dev)
    if c["op"] == "attend":
        s["q"] = normal(B, T, c["Hq"], D)
        if c["K"]:  # blocks that begin at or before the query, all different, ascending, -1 where there are fewer
            M = -(-n // 64)
            last = (ns.long()[:, None] - T + torch.arange(T, device=dev)) // 64  # a query's own block
            own_block = last[:, None, :, None]
            x = torch.rand(B, Hkv, T, M, generator=g, device=dev)
            x = torch.where(torch.arange(M, device=dev) <= own_block, x, -1.0)
            top, at = x.topk(min(c["K"], M), dim=-1)
            at = torch.where(top >= 0, at, 1 << 30).sort(-1).values
            at = torch.where(at < (1 << 30), at, -1)
            s["idx"] = torch.nn.functional.pad(at, (0, c["K"] - at.shape[-1]), value=-1).to(torch.int32)
        s["out_dtype"] = torch.bfloat16 if c["out"] == "bf16" else torch.float32
    if own:  # the descriptor and the scratch that a decoding program makes once and keeps
        import pyramid_top_block_gb300 as pisa
        s["cache"] = pisa.PagedCache(s["pages"], s["table"], P)
        s["workspace"] = pisa.cache_workspace(s["cache"])
        if c["op"] == "attend":
            s["buffer"] = torch.empty(B, T, c["Hq"], D, dtype=s["out_dtype"], device=dev)
    return s


def rotated(x, cos, sin, rot, interleaved):
    """bf16 x [B, T, H, 64] turned by cos, sin [B, T, 1, rot / 2] in its first rot dims; rounded once, from 64 bits."""
    y = x[..., :rot].double()
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else y.chunk(2, -1)
    c, s = cos.double(), sin.double()
    a, b = a * c - b * s, b * c + a * s
    y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y.to(torch.bfloat16), x[..., rot:]], -1)


def _plain_append(s):
    B, T, rot = s["B"], s["T"], s["rot"]
    t = torch.arange(T, device=s["q"].device)
    there = t < s["counts"][:, None]
    b, t = there.nonzero(as_tuple=True)
    pos = s["start"].long()[b] + t
    cos, sin = s["rotary"][pos].chunk(2, -1)
    q = rotated(s["q"][b, t], cos[:, None], sin[:, None], rot, s["interleaved"])
    k = rotated(s["k"][b, t], cos[:, None], sin[:, None], rot, s["interleaved"])
    s["q_out"][b, t], s["k_out"][b, t] = q, k
    page, rec, row = places(s, b, pos)
    v = s["v"][b, t]
    if s["kind"] == "bf16":
        kp, vp = views(s)
        kp[page, :, rec, row], vp[page, :, rec, row] = k, v
        return s["q_out"], s["k_out"], s["pages"]
    kc, ks, vc, vs = views(s)
    kc[page, :, rec, row], ks[page, :, rec, row] = quantised(k.float())
    vc[page, :, rec, row], vs[page, :, rec, row] = quantised(v.float())
    return (s["q_out"], s["k_out"]) + _plain_read(s)


def _fetch(s, page, head, rec, row):
    """fp32 keys and values at places that broadcast together."""
    if s["kind"] == "bf16":
        kp, vp = views(s)
        return kp[page, head, rec, row].float(), vp[page, head, rec, row].float()
    kc, ks, vc, vs = views(s)
    at = (page, head, rec, row)
    return dequantised(kc[at], ks[at]), dequantised(vc[at], vs[at])


def _plain_read(s):
    t = torch.arange(s["T"], device=s["table"].device)
    b, t = (t < s["counts"][:, None]).nonzero(as_tuple=True)
    page, rec, row = places(s, b, s["start"].long()[b] + t)
    head = torch.arange(s["Hkv"], device=t.device)
    k, v = _fetch(s, page[:, None], head, rec[:, None], row[:, None])
    s["k_read"][b, t], s["v_read"][b, t] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    return s["k_read"], s["v_read"]


def _plain_attend(s):
    B, T, Hkv, Hq, n = s["B"], s["T"], s["Hkv"], s["Hq"], s["n"]
    dev, G = s["q"].device, s["Hq"] // s["Hkv"]
    q = s["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4)  # [B, Hkv, T, G, 64]
    at = s["lengths"].long()[:, None] - T + torch.arange(T, device=dev)  # position of each query
    b = torch.arange(B, device=dev)
    if s["K"]:  # the tokens of the listed blocks, a query's own set each
        pos = s["idx"].long()[..., None] * 64 + torch.arange(64, device=dev)
        pos = torch.where(s["idx"][..., None] >= 0, pos, 1 << 30).flatten(-2)  # [B, Hkv, T, K * 64]
        seen = pos <= at[:, None, :, None]
        pos = torch.where(seen, pos, 0)
        page, rec, row = places(s, b[:, None, None, None], pos)
        head = torch.arange(Hkv, device=dev)[:, None, None]
        k, v = _fetch(s, page, head, rec, row)  # [B, Hkv, T, K * 64, 64]
        x = q @ k.transpose(-1, -2)
    else:  # every token of the sequence, shared by its queries
        pos = torch.arange(n, device=dev)
        seen = (pos <= at[..., None])[:, None]  # [B, 1, T, n]
        page, rec, row = places(s, b[:, None], pos.expand(B, n))
        head = torch.arange(Hkv, device=dev)[:, None]
        k, v = _fetch(s, page[:, None], head, rec[:, None], row[:, None])  # [B, Hkv, n, 64]
        x = (q.flatten(2, 3) @ k.transpose(-1, -2)).unflatten(2, (T, G))
    x = torch.where(seen[..., None, :], x * 0.125, -math.inf)  # [B, Hkv, T, G, keys]
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    o = e @ v if s["K"] else (e.flatten(2, 3) @ v).unflatten(2, (T, G))
    o = o / e.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(s["out_dtype"])


def _own_append(s):
    import pyramid_top_block_gb300 as pisa
    cache = s["cache"]
    q, k = pisa.cache_append(s["q"], s["k"], s["v"], cache, s["start"], s["rotary"], counts=s["counts"],
                             interleaved=s["interleaved"], q_out=s["q_out"], k_out=s["k_out"])
    if s["kind"] == "bf16":
        return q, k, s["pages"]
    return (q, k) + _own_read(s)


def _own_read(s):
    import pyramid_top_block_gb300 as pisa
    return pisa.cache_read(s["cache"], s["start"], s["T"], counts=s["counts"], k_out=s["k_read"], v_out=s["v_read"])


def _own_attend(s):
    import pyramid_top_block_gb300 as pisa
    return pisa.cache_attention(s["q"], s["cache"], s["lengths"], idx=s.get("idx"), out=s["buffer"],
                                workspace=s["workspace"])


def run(s):
    if own:
        return {"append": _own_append, "attend": _own_attend, "read": _own_read}[s["op"]](s)
    return {"append": _plain_append, "attend": _plain_attend, "read": _plain_read}[s["op"]](s)


# The definition in 64 bits, one sequence after the other.


def _power(e):
    """2^e, exactly (the device's pow need not be), for whole e of -128..127 as float64."""
    return torch.tensor([2.0 ** i for i in range(-128, 128)], dtype=torch.float64, device=e.device)[e.long() + 128]


def _exact_value(codes, scales):
    """e2m1 x e4m3 by their fields: codes [..., 32], scales [..., 4] -> float64 [..., 64]."""
    c = torch.empty(codes.shape[:-1] + (64,), dtype=torch.int64, device=codes.device)
    c[..., 0::2], c[..., 1::2] = (codes % 16).long(), (codes // 16).long()
    e, m = (c >> 1) & 3, (c & 1).double()
    x = torch.where(e == 0, m * 0.5, (1 + m / 2) * _power(e - 1))
    x = torch.where(c >= 8, -x, x)
    z = scales.long()
    ze, zm = (z >> 3) & 15, (z & 7).double()
    f = torch.where(ze == 0, zm * 2.0 ** -9, (1 + zm / 8) * _power(ze - 7))
    return x * f.repeat_interleave(16, dim=-1)


def _exact_tokens(s, b, pos):
    """float64 K, V [len(pos), Hkv, 64] of sequence b."""
    P, U = s["page"], min(s["page"], 64)
    record = s["table"][b].long()[pos // P] * (P // U) * s["Hkv"] + (pos % P) // U
    record = record[:, None] + torch.arange(s["Hkv"], device=pos.device) * (P // U)  # records lie page, head, part
    flat = s["pages"].reshape((-1,) + tuple(s["pages"].shape[3:]))
    u = (pos % U)[:, None]
    if s["kind"] == "bf16":
        return flat[record, 0, u].double(), flat[record, 1, u].double()

    def part(begin, width):
        return flat[record[..., None], begin + u[..., None] * width + torch.arange(width, device=pos.device)]

    return (_exact_value(part(0, 32), part(32 * U, 4)), _exact_value(part(36 * U, 32), part(68 * U, 4)))


def _exact_round(x):
    """The values that 64-wide rows of float64 x have in the cache's 4 bits."""
    y = x.reshape(x.shape[:-1] + (4, 16))
    top = y.abs().amax(-1) / 6
    e = torch.frexp(top.clamp(min=2.0 ** -60)).exponent - 1  # top lies in [2^e, 2^(e + 1))
    step = _power(e.clamp(min=-6) - 3)
    f = (torch.round(top / step) * step).clamp(max=448.0)[..., None]  # e4m3: three bits below the leading one
    r = y.abs() / torch.where(f > 0, f, 1.0)
    grid = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0))  # e2m1: one bit below the leading one
    v = (torch.round(r / grid) * grid).clamp(max=6.0) * f
    return torch.where(y < 0, -v, v).reshape(x.shape)


def _exact_turn(x, cos, sin, rot, interleaved):
    y = x.double().clone()
    i = torch.arange(rot // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., a] = x[..., a].double() * cos - x[..., b].double() * sin
    y[..., b] = x[..., a].double() * sin + x[..., b].double() * cos
    return y


def exact(case, seed):
    if case["op"] == "attend" and case["B"] * case["T"] * case["Hkv"] > 4096:
        return None  # too many separate softmaxes for the loop below
    s = prepare(case, seed)
    dev = s["table"].device
    B, T, Hkv = s["B"], s["T"], s["Hkv"]
    if s["op"] == "attend":
        G = s["Hq"] // Hkv
        out = torch.zeros(B, T, s["Hq"], D, dtype=torch.float64, device=dev)
        for b in range(B):
            n = int(s["lengths"][b])
            if not s["K"]:
                k, v = _exact_tokens(s, b, torch.arange(n, device=dev))
            for t in range(T):
                p = n - T + t
                if p < 0:
                    continue
                for h in range(Hkv):
                    if s["K"]:
                        blocks = s["idx"][b, h, t]
                        blocks = blocks[blocks >= 0].long()
                        pos = (blocks[:, None] * 64 + torch.arange(64, device=dev)).flatten()
                        kk, vv = (x[:, h] for x in _exact_tokens(s, b, pos[pos <= p]))
                    else:
                        kk, vv = k[:p + 1, h], v[:p + 1, h]
                    z = s["q"][b, t, h * G:(h + 1) * G].double() @ kk.T / 8
                    out[b, t, h * G:(h + 1) * G] = torch.softmax(z, -1) @ vv
        return out
    if s["op"] == "read":
        k_read, v_read = s["k_read"].double(), s["v_read"].double()
        for b in range(B):
            m = int(s["counts"][b])
            k_read[b, :m], v_read[b, :m] = _exact_tokens(s, b, int(s["start"][b]) + torch.arange(m, device=dev))
        return k_read, v_read
    q_out, k_out = s["q_out"].double(), s["k_out"].double()
    pages = s["pages"].double() if s["kind"] == "bf16" else None
    k_read, v_read = torch.zeros_like(k_out), torch.zeros_like(k_out)
    U = min(s["page"], 64)
    for b in range(B):
        m = int(s["counts"][b])
        pos = int(s["start"][b]) + torch.arange(m, device=dev)
        cos, sin = (x[:, None].double() for x in s["rotary"][pos].chunk(2, -1))
        q_out[b, :m] = _exact_turn(s["q"][b, :m], cos, sin, s["rot"], s["interleaved"])
        k = _exact_turn(s["k"][b, :m], cos, sin, s["rot"], s["interleaved"])
        k_out[b, :m] = k
        v = s["v"][b, :m].double()
        if pages is None:  # the cache holds what the keys are in bf16, in 4 bits
            k_read[b, :m], v_read[b, :m] = _exact_round(k.to(torch.bfloat16).double()), _exact_round(v)
        else:
            page, part, u = s["table"][b].long()[pos // s["page"]], pos % s["page"] // U, pos % U
            pages[page, :, part, 0, u], pages[page, :, part, 1, u] = k, v
    return (q_out, k_out, pages) if pages is not None else (q_out, k_out, k_read, v_read)
