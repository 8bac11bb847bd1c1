"""What prompts, capped and biased scores, and shared pages cost on the paged cache: cases, inputs, plain forms, and
the framework's own calls.

Five operators around one paged KV cache:

* ``append``: rotate new queries and keys whose positions have several axes (time, height, width of an image or a
  video) and put keys and values into the cache;
* ``prompt``: the tokens of a prompt, or of a chunk of one, attend over the cache, each over its own span of it
  (causal, a window, documents, a prefix that is seen from both sides), with capped scores or a bias by distance;
* ``token``: the newest tokens of each sequence attend over the cache with a window, capped scores or such a bias;
* ``branch``: sequences become copies of others by sharing their pages (parallel samples, beams), then pages for the
  next tokens are reserved, and a shared page that is about to be written is copied;
* ``compact``: the pages in use move to the front of the pool, so that its end can be given back.

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
        # one decoding step behind prompts with images: rotation by three axes, a batch of long contexts
        dict(name="append step 16 3 axes 4-bit", op="append", kind="e2m1", B=16, T=1, n=131072, Hq=32, Hkv=2, page=64,
             rot=64, interleaved=False, axes=3, mixed=False, ragged=False),
        # a whole prompt of images and text, the latency benchmark's 32K size
        dict(name="append prompt 32768 3 axes bf16", op="append", kind="bf16", B=1, T=32768, n=32768, Hq=32, Hkv=2,
             page=64, rot=64, interleaved=False, axes=3, mixed=True, ragged=False),
        # a decoding step of a layer with capped scores over long contexts (the decode benchmark's sizes)
        dict(name="token 16x131072 cap 4-bit", op="token", kind="e2m1", B=16, T=1, n=131072, Hq=32, Hkv=2, page=64,
             cap=30.0, slopes=False, window=0, ragged=False),
        # a decoding step of a layer that sees a window of its context, many short sequences
        dict(name="token 65x16421 window 1024 bf16", op="token", kind="bf16", B=65, T=1, n=16421, Hq=16, Hkv=4,
             page=16, cap=0.0, slopes=False, window=1024, ragged=True),
        # three speculative tokens of a model with a bias by distance, long ragged contexts
        dict(name="token 8x131072 T=3 slopes bf16", op="token", kind="bf16", B=8, T=3, n=131072, Hq=16, Hkv=2,
             page=64, cap=0.0, slopes=True, window=0, ragged=True),
        # a packed prompt of several documents, the smallest configuration's sizes
        dict(name="prompt 2048 documents bf16", op="prompt", kind="bf16", B=1, T=2048, n=2048, Hq=4, Hkv=1, page=64,
             cap=0.0, slopes=False, window=0, spans="documents", ragged=False),
        # two whole prompts of different lengths, capped scores (the ragged benchmark's size)
        dict(name="prompt 2x16421 cap bf16", op="prompt", kind="bf16", B=2, T=16421, n=16421, Hq=32, Hkv=2, page=128,
             cap=30.0, slopes=False, window=0, spans="causal", ragged=True),
        # a chunk of a long prompt over all that is already cached
        dict(name="prompt 2048 at 131072 4-bit", op="prompt", kind="e2m1", B=1, T=2048, n=131072, Hq=32, Hkv=2,
             page=64, cap=0.0, slopes=False, window=0, spans="causal", ragged=False),
        # sixteen prompts sampled four times each, then pages for the next token of each
        dict(name="branch 64 of 16x2048", op="branch", B=64, n=2048, page=64, Hkv=2, layers=1, T=1, samples=4),
        # a reordering of beams of many layers, where each beam's last page is copied
        dict(name="branch 256 of 32x1201 16 layers", op="branch", B=256, n=1201, page=64, Hkv=2, layers=16, T=8,
             samples=8),
        # a pool with holes after half of the short sequences have ended
        dict(name="compact 64x2049", op="compact", B=64, n=2049, page=16, Hkv=4, layers=1, gone=0.5),
        # the same for long sequences of several layers
        dict(name="compact 32x16421 4 layers", op="compact", B=32, n=16421, page=64, Hkv=2, layers=4, gone=0.6),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "token", "token", "prompt", "prompt", "branch", "compact"])
    c = dict(op=op, page=rng.choice([16, 32, 64, 128, 256]), Hkv=rng.choice([1, 2, 4, 8]))
    if op == "branch":
        c.update(B=_spread(rng, 2, 512), layers=rng.choice([1, 2, 4, 8]), T=_spread(rng, 1, 64),
                 samples=rng.choice([1, 2, 4, 8]))
        page_bytes = c["layers"] * c["Hkv"] * c["page"] * 256
        c["n"] = _spread(rng, 1, max(2, min(16384, (1 << 29) // page_bytes * c["page"] // c["B"])))
        return c
    if op == "compact":
        c.update(B=_spread(rng, 1, 256), layers=rng.choice([1, 2, 4, 8]), gone=rng.uniform(0.05, 0.9))
        page_bytes = c["layers"] * c["Hkv"] * c["page"] * 256
        c["n"] = _spread(rng, 1, max(2, min(131072, (1 << 30) // page_bytes * c["page"] // c["B"])))
        return c
    c.update(kind=rng.choice(["bf16", "e2m1"]), ragged=rng.random() < 0.6)
    G = rng.choice([1, 2, 4, 8, 16])
    c["Hq"] = G * c["Hkv"]
    if op == "append":
        c["B"] = _spread(rng, 1, 128)
        most = 900000 // (c["B"] * (c["Hq"] + 4 * c["Hkv"] + 8))
        c["T"] = 1 if rng.random() < 0.4 else _spread(rng, 2, max(2, min(most, 32768)))
        c.update(n=c["T"] + _spread(rng, 1, 131072 // c["B"]), rot=rng.choice([16, 32, 48, 64, 64]),
                 interleaved=rng.random() < 0.5, axes=rng.choice([1, 2, 3, 3, 4]), mixed=rng.random() < 0.5)
        return c
    c.update(cap=rng.choice([0.0, 0.0, 20.0, 50.0]), slopes=rng.random() < 0.3)
    c["window"] = _spread(rng, 1, 8192) if rng.random() < 0.4 else 0
    if op == "token":
        c["B"] = _spread(rng, 1, 128)
        c["T"] = 1 if rng.random() < 0.6 else rng.randint(2, 16)
        rows = c["B"] * c["Hkv"] * c["T"]
        most = (1 << 22) // rows if c["kind"] == "e2m1" else (1 << 20) // rows
        c["n"] = max(c["T"], _spread(rng, 1, max(1, min(262144, most))))
        return c
    c["B"] = _spread(rng, 1, 16)
    c["T"] = _spread(rng, 1, max(1, 16384 // c["B"]))
    most = (1 << 32) // (c["B"] * c["Hq"] * c["T"])  # logits of the largest listed case, at most
    c["n"] = c["T"] + (0 if rng.random() < 0.4 else _spread(rng, 1, max(1, min(131072, most))))
    c["spans"] = rng.choice(["causal", "causal", "documents", "prefix"])
    while c["B"] * c["Hq"] * c["T"] * c["n"] > (1 << 33):
        c["T"] = c["n"] = max(1, c["T"] // 2)
    return c


def lengths_of(c):
    """Tokens of each sequence after the case's call: n, or between 1 and n where the case is ragged."""
    if not c["ragged"]:
        return [c["n"]] * c["B"]
    r = random.Random(1000003 * c["B"] + c["n"])
    return [c["n"] if b == 0 else max(1, int(c["n"] * r.uniform(0.05, 1.0))) for b in range(c["B"])]


def counts_of(c):
    """New tokens of each sequence: at most T, and no more than there are."""
    return [min(c["T"], n) for n in lengths_of(c)]


def row_bytes(c):
    """Bytes of one token's keys and values of one KV head."""
    return 256 if c["kind"] == "bf16" else 72


def spans_of(c):
    """(first, last) of each new token, as lists of B lists of counts numbers: it sees the cached tokens
    first .. last - 1."""
    r = random.Random(7 + c["T"])
    out = []
    for n, m in zip(lengths_of(c), counts_of(c)):
        start = n - m
        p = list(range(start, n))
        first, last = [0] * m, [x + 1 for x in p]
        if c["spans"] == "documents":  # of about 300 tokens; the earlier tokens belong to the first one
            at = 0
            for i, x in enumerate(p):
                if i and r.random() < 1 / 300:
                    at = x
                first[i] = at
        elif c["spans"] == "prefix":  # the first third of what is new is seen from both sides
            edge = start + (m + 2) // 3
            last = [max(x, edge) for x in last]
        if c["window"]:
            first = [max(f, x - c["window"] + 1) for f, x in zip(first, p)]
        out.append((first, last))
    return out


def sequences_of(c):
    """Lengths of the sequences that hold pages before a branch or a compaction."""
    held = c["B"] // c["samples"] if c["op"] == "branch" else c["B"]
    r = random.Random(31 * c["B"] + c["n"])
    return [c["n"] if b == 0 else max(1, int(c["n"] * r.uniform(0.4, 1.0))) for b in range(max(1, held))]


def plan_of(c, seed=0):
    """A pool's state as whole numbers: pages in all, table rows, references and lengths, and for a branch the
    parent of every sequence."""
    r = random.Random(seed * 7919 + 13)
    P, ns = c["page"], sequences_of(c)
    per = [-(-n // P) for n in ns]
    wide = max(per) + -(-c.get("T", 0) // P) + 1
    B = max(c["B"], len(ns))
    if c["op"] == "branch":
        total = sum(per) + B * (2 + -(-c["T"] // P))
    else:
        total = sum(per) + 3
    order = list(range(total))
    r.shuffle(order)
    table, refs, lengths, at = [], [0] * total, [], 0
    for b in range(B):
        row = [-1] * wide
        if b < len(ns) and not (c["op"] == "compact" and len(ns) > 1 and r.random() < c["gone"]):
            row[:per[b]] = order[at:at + per[b]]
            for x in row[:per[b]]:
                refs[x] += 1
        lengths.append(ns[b] if row[0] >= 0 else 0)
        at += per[b] if b < len(ns) else 0
        table.append(row)
    # the samples of a prompt side by side; a few sequences end
    parents = [-1 if r.random() < 0.02 else min(b // c["samples"], len(ns) - 1) for b in range(B)] \
        if c["op"] == "branch" else None
    return total, wide, table, refs, lengths, parents


def _page_values(c):
    return c["layers"] * c["Hkv"] * c["page"] * 2 * D


def work(case):
    c = case
    if c["op"] in ("branch", "compact"):
        total, wide, table, refs, lengths, parents = plan_of(c)
        page = 2 * _page_values(c)
        if c["op"] == "compact":
            used = sum(x > 0 for x in refs)
            moved = sum(x > 0 for x in refs[used:])
            return dict(bytes=2 * moved * page + 8 * total + 4 * wide * len(table), flops=0)
        kids = [sum(q == b for q in parents) for b in range(len(table))]
        copied = sum(1 for q in parents if q >= 0 and kids[q] > 1 and lengths[q] % c["page"])
        return dict(bytes=2 * copied * page + 4 * total + 8 * wide * len(table), flops=0)
    ns, per = lengths_of(c), row_bytes(c)
    if c["op"] == "append":
        tok = sum(counts_of(c))
        heads = c["Hq"] + c["Hkv"]
        # queries, keys and values in; rotated queries and keys and the pages out; positions and angles of a token
        moved = tok * ((2 * heads + c["Hkv"]) * 2 * D + c["Hkv"] * per + 4 * c["rot"] + 4 * c["axes"])
        if c["kind"] == "e2m1":  # and the values that the new codes stand for
            moved += tok * c["Hkv"] * (per + 4 * D)
        return dict(bytes=moved, flops=3 * c["rot"] * heads * tok)
    G, T = c["Hq"] // c["Hkv"], c["T"]
    if c["op"] == "token":
        p = [[n - T + t for t in range(T)] for n in ns]
        lo = [[max(0, x - c["window"] + 1) if c["window"] else 0 for x in q] for q in p]
        seen = sum(max(0, x + 1 - f) for q, fs in zip(p, lo) for x, f in zip(q, fs))
        read = sum(max(0, q[-1] + 1 - fs[0]) for q, fs in zip(p, lo))
        return dict(bytes=read * c["Hkv"] * per + 4 * D * c["B"] * T * c["Hq"], flops=4 * D * c["Hq"] * seen)
    spans = spans_of(c)
    seen = sum(max(0, y - x) for f, l in spans for x, y in zip(f, l))
    read = sum(max(l) - min(f) for f, l in spans)
    return dict(bytes=read * c["Hkv"] * per + 4 * D * sum(counts_of(c)) * c["Hq"], flops=4 * D * c["Hq"] * seen)


def quantised(x):
    """float [..., 64] -> (codes uint8 [..., 32], scales uint8 [..., 4]): one e4m3 scale per 16 values, the largest
    of them at 6; nearest code, a value half way between two to the even code, past the largest the largest."""
    y = x.unflatten(-1, (4, 16))
    scale = (y.abs().amax(-1).double() / 6).clamp(max=448.0).float().to(E4M3)
    s = scale.float().unsqueeze(-1)
    r = y.abs().double() / torch.where(s > 0, s, 1.0).double()
    borders = torch.tensor([(a + b) / 2 for a, b in zip(MAGNITUDES, MAGNITUDES[1:])], dtype=torch.float64,
                           device=x.device)
    # the border between codes i and i + 1 goes to the even one
    above, at = torch.bucketize(r, borders), torch.bucketize(r, borders, right=True)
    code = torch.where(at % 2 == 0, at, above).to(torch.uint8)
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


def _prepare_pool(c, seed):
    dev = "cuda"
    total, wide, table, refs, lengths, parents = plan_of(c, seed)
    B, U = len(table), min(c["page"], 64)
    g = torch.Generator(device=dev).manual_seed(seed)
    s = dict(c, B=B, n_pages=total, wide=wide)
    shape = (total, c["layers"], c["Hkv"], c["page"] // U, 2, U, D)
    s["pages"] = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    s["pages"].normal_(generator=g)
    # one buffer, so that a pass begins by putting all of it back with one copy
    s["before"] = torch.tensor(sum(table, []) + refs + lengths, dtype=torch.int32, device=dev)
    s["meta"] = s["before"].clone()
    t, r, n = s["meta"].split([B * wide, total, B])
    s["table"], s["refs"], s["lengths"] = t.view(B, wide), r, n
    if c["op"] == "branch":
        s["parents"] = torch.tensor(parents, dtype=torch.int32, device=dev)
        s["granted"] = torch.zeros(B, dtype=torch.int32, device=dev)
    else:
        s["used"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if own:  # the handle and the scratch that a serving program makes once and keeps
        import pyramid_top_block_gb300 as pisa
        s["pool"] = pisa.PagePool(s["pages"], s["table"], s["refs"], c["page"])
        s["workspace"] = pisa.pool_workspace(s["pool"])
    return s


def prepare(case, seed):
    c = dict(case)
    if c["op"] in ("branch", "compact"):
        return _prepare_pool(c, seed)
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
    if c["op"] != "token":
        s["counts"] = torch.tensor(counts_of(c), dtype=torch.int32, device=dev)
        s["start"] = ns - s["counts"]
    if c["op"] == "append":
        # the three projections of one fused product, side by side in a token's row
        qkv = normal(B, T, c["Hq"] + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv.split([c["Hq"], Hkv, Hkv], dim=2)
        s["k"] *= k_scale.to(torch.bfloat16)
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
        angle = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * inv
        s["rotary"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        # images of 24 x 32 patches between runs of text, where the axes go together
        at = s["start"][:, None].long() + torch.arange(T, device=dev)
        patch = at % 1024
        in_image = (patch < 768) & (at >= 1024)
        axes = torch.stack([at, at - patch + patch // 32, at - patch + patch % 32, patch])[:c["axes"]]
        s["positions"] = torch.where(in_image, axes, at).clamp(0, n - 1).to(torch.int32).contiguous()
        half = c["rot"] // 2
        s["axes"] = tuple(i % c["axes"] if c["mixed"] else i * c["axes"] // half for i in range(half))
        s["q_out"] = torch.zeros(B, T, c["Hq"], D, dtype=torch.bfloat16, device=dev)
        s["k_out"] = torch.zeros(B, T, Hkv, D, dtype=torch.bfloat16, device=dev)
        if c["kind"] == "e2m1":
            s["k_read"] = torch.zeros(B, T, Hkv, D, dtype=torch.bfloat16, device=dev)
            s["v_read"] = torch.zeros(B, T, Hkv, D, dtype=torch.bfloat16, device=dev)
    else:
        s["q"] = normal(B, T, c["Hq"], D, scale=3.0 if c["cap"] else 1.0)  # (logits that the cap bends)
        s["buffer"] = torch.zeros(B, T, c["Hq"], D, dtype=torch.bfloat16, device=dev)
        s["slope"] = None
        if c["slopes"]:
            s["slope"] = torch.tensor([2.0 ** (-8 * (h + 1) / c["Hq"]) for h in range(c["Hq"])], device=dev)
    if c["op"] == "prompt":
        s["first"], s["last"] = torch.zeros(2, B, T, dtype=torch.int32, device=dev)
        for b, (f, l) in enumerate(spans_of(dict(c, window=0))):
            s["first"][b, :len(f)] = torch.tensor(f, dtype=torch.int32, device=dev)
            s["last"][b, :len(l)] = torch.tensor(l, dtype=torch.int32, device=dev)
        if c["spans"] != "documents":
            s["first"] = None
        if c["spans"] != "prefix":
            s["last"] = None
    if own:  # the descriptor and the scratch that a serving program makes once and keeps
        import pyramid_top_block_gb300 as pisa
        s["cache"] = pisa.PagedCache(s["pages"], s["table"], P)
        s["workspace"] = pisa.cache_workspace(s["cache"])
    return s


def rotated(x, cos, sin, rot, interleaved):
    """bf16 x [..., H, 64] turned by cos, sin [..., 1, rot / 2] in its first rot dims; rounded once, from 64 bits."""
    y = x[..., :rot].double()
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else y.chunk(2, -1)
    c, s = cos.double(), sin.double()
    a, b = a * c - b * s, b * c + a * s
    y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y.to(torch.bfloat16), x[..., rot:]], -1)


def _plain_append(s):
    B, T, rot = s["B"], s["T"], s["rot"]
    t = torch.arange(T, device=s["q"].device)
    b, t = (t < s["counts"][:, None]).nonzero(as_tuple=True)
    axis = torch.tensor(s["axes"], device=t.device)
    at = s["positions"][:, b, t].long()[axis].T  # [tokens, rot / 2]: the position each pair turns by
    i = torch.arange(rot // 2, device=t.device)
    cos, sin = s["rotary"][at, i], s["rotary"][at, rot // 2 + i]
    q = rotated(s["q"][b, t], cos[:, None], sin[:, None], rot, s["interleaved"])
    k = rotated(s["k"][b, t], cos[:, None], sin[:, None], rot, s["interleaved"])
    s["q_out"][b, t], s["k_out"][b, t] = q, k
    page, rec, row = places(s, b, s["start"].long()[b] + t)
    v = s["v"][b, t]
    if s["kind"] == "bf16":
        kp, vp = views(s)
        kp[page, :, rec, row], vp[page, :, rec, row] = k, v
        return s["q_out"], s["k_out"], s["pages"]
    kc, ks, vc, vs = views(s)
    kc[page, :, rec, row], ks[page, :, rec, row] = quantised(k.float())
    vc[page, :, rec, row], vs[page, :, rec, row] = quantised(v.float())
    head = torch.arange(s["Hkv"], device=t.device)
    k, v = _fetch(s, page[:, None], head, rec[:, None], row[:, None])
    s["k_read"][b, t], s["v_read"][b, t] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    return s["q_out"], s["k_out"], s["k_read"], s["v_read"]


def _fetch(s, page, head, rec, row):
    """fp32 keys and values at places that broadcast together."""
    if s["kind"] == "bf16":
        kp, vp = views(s)
        return kp[page, head, rec, row].float(), vp[page, head, rec, row].float()
    kc, ks, vc, vs = views(s)
    at = (page, head, rec, row)
    return dequantised(kc[at], ks[at]), dequantised(vc[at], vs[at])


def _keys(s, base, width):
    """Positions base[b] .. + width - 1 of every sequence (held at 0 and n - 1), their keys and values
    [B, Hkv, width, 64]."""
    dev = s["q"].device
    pos = (base[:, None] + torch.arange(width, device=dev)).clamp(0, s["n"] - 1)
    page, rec, row = places(s, torch.arange(s["B"], device=dev)[:, None], pos)
    head = torch.arange(s["Hkv"], device=dev)[:, None]
    k, v = _fetch(s, page[:, None], head, rec[:, None], row[:, None])
    return k, v


def _weighted(s, q, k, v, at, lo, hi, base):
    """Attention of q [B, t, Hq, 64] at positions at [B, t] over keys at base[b] + 0, 1, .., each seeing lo .. hi - 1."""
    B, t, Hq, _ = q.shape
    G = Hq // s["Hkv"]
    x = q.float().view(B, t, s["Hkv"], G, D).permute(0, 2, 1, 3, 4).flatten(2, 3) @ k.transpose(-1, -2)
    x = x.unflatten(2, (t, G)) * 0.125  # [B, Hkv, t, G, keys]
    pos = base[:, None] + torch.arange(k.shape[2], device=q.device)
    seen = (pos[:, None] >= lo[..., None]) & (pos[:, None] < hi[..., None])  # [B, t, keys]
    if s["cap"]:
        x = s["cap"] * torch.tanh(x / s["cap"])
    if s["slope"] is not None:
        far = (at[..., None] - pos[:, None]).abs().float()  # (exact)
        x = x - s["slope"].view(s["Hkv"], 1, G, 1) * far[:, None, :, None]
    x = torch.where(seen[:, None, :, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    o = (e.flatten(2, 3) @ v).unflatten(2, (t, G)) / e.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.permute(0, 2, 1, 3, 4).reshape(B, t, Hq, D).to(torch.bfloat16)


def _plain_token(s):
    T, W = s["T"], s["window"]
    at = s["lengths"].long()[:, None] - T + torch.arange(T, device=s["q"].device)
    lo = (at - W + 1 if W else at * 0).clamp(min=0)
    width = min(s["n"], W + T - 1) if W else s["n"]
    base = (at[:, -1] + 1 - width).clamp(min=0) if W else at[:, 0] * 0
    k, v = _keys(s, base, width)
    s["buffer"].copy_(_weighted(s, s["q"], k, v, at, lo, at + 1, base))
    return s["buffer"]


def _plain_prompt(s):
    B, T = s["B"], s["T"]
    t = torch.arange(T, device=s["q"].device)
    at = s["start"].long()[:, None] + t
    lo = at * 0 if s["first"] is None else s["first"].long()
    lo = torch.maximum(lo, at - s["window"] + 1) if s["window"] else lo
    hi = at + 1 if s["last"] is None else s["last"].long()
    base = torch.zeros(B, dtype=torch.long, device=t.device)
    k, v = _keys(s, base, s["n"])
    there = t < s["counts"][:, None]
    step = max(1, (1 << 29) // (B * s["Hq"] * s["n"]))
    for i in range(0, T, step):  # (all of the logits at once would not fit)
        j = slice(i, i + step)
        o = _weighted(s, s["q"][:, j], k, v, at[:, j], lo[:, j], hi[:, j], base)
        s["buffer"][:, j] = torch.where(there[:, j, None, None], o, s["buffer"][:, j])
    return s["buffer"]


def _plain_branch(s):
    s["meta"].copy_(s["before"])
    table, refs, lengths, P, n_pages = s["table"], s["refs"], s["lengths"], s["page"], s["n_pages"]

    def count(entries):
        e = entries[(entries >= 0) & (entries < n_pages)].long()
        return torch.bincount(e, minlength=n_pages).to(torch.int32)

    # every sequence takes its parent's row; one without a parent lets its pages go
    q = s["parents"].long()
    new = torch.where(q[:, None] >= 0, table[q.clamp(min=0)], -1)
    refs += count(new) - count(table)
    table.copy_(new)
    lengths.copy_(torch.where(q >= 0, lengths[q.clamp(min=0)], 0))
    # pages for the next T tokens: fresh ones, lowest number first, for those that are missing or shared
    n, e = lengths.long(), torch.arange(s["wide"], device=q.device)
    fits = (n >= 0) & (n + s["T"] <= s["wide"] * P)
    written = (e >= (n // P)[:, None]) & (e < ((n + s["T"] + P - 1) // P)[:, None])
    held = (table >= 0) & (table < n_pages)
    old = torch.where(held, table, 0).long()
    shared = held & (refs[old] > 1)
    take = written & (~held | shared) & fits[:, None]
    need = take.sum(1)
    free = (refs == 0).nonzero()[:, 0]
    served = fits & ((need == 0) | (need.cumsum(0) <= free.numel()))
    take &= served[:, None]
    b, i = take.nonzero(as_tuple=True)
    fresh = free[:b.numel()]
    gone = old[b, i][shared[b, i]]
    copied = shared[b, i] & (i == n[b] // P) & (n[b] % P > 0)
    s["pages"][fresh[copied]] = s["pages"][old[b, i][copied]]
    refs -= torch.bincount(gone, minlength=n_pages).to(torch.int32)
    refs[fresh] = 1
    table[b, i] = fresh.to(torch.int32)
    s["granted"].copy_(torch.where(served, s["T"], 0))
    return table, refs, lengths, s["granted"], s["pages"]


def _plain_compact(s):
    s["meta"].copy_(s["before"])
    table, refs = s["table"], s["refs"]
    at = (refs != 0).nonzero()[:, 0]
    used = at.numel()
    src = at[at >= used]
    dst = (refs[:used] == 0).nonzero()[:, 0]
    s["pages"][dst] = s["pages"][src]
    to = torch.arange(s["n_pages"], device=refs.device)
    to[src] = dst
    held = (table >= 0) & (table < s["n_pages"])
    table.copy_(torch.where(held, to[torch.where(held, table, 0).long()].to(torch.int32), table))
    refs[dst] = refs[src]
    refs[src] = 0
    s["used"].fill_(used)
    return table, refs, s["used"], s["pages"]


def _own(s):
    import pyramid_top_block_gb300 as pisa
    if s["op"] == "append":
        q, k = pisa.cache_append(s["q"], s["k"], s["v"], s["cache"], s["start"], s["rotary"], counts=s["counts"],
                                 interleaved=s["interleaved"], q_out=s["q_out"], k_out=s["k_out"],
                                 workspace=s["workspace"], positions=s["positions"], axes=s["axes"])
        if s["kind"] == "bf16":
            return q, k, s["pages"]
        return (q, k) + pisa.cache_read(s["cache"], s["start"], s["T"], counts=s["counts"], k_out=s["k_read"],
                                        v_out=s["v_read"], workspace=s["workspace"])
    if s["op"] == "token":
        return pisa.cache_attention(s["q"], s["cache"], s["lengths"], out=s["buffer"], workspace=s["workspace"],
                                    cap=s["cap"], slopes=s["slope"], window=s["window"])
    if s["op"] == "prompt":
        return pisa.cache_prompt_attention(s["q"], s["cache"], s["start"], counts=s["counts"], out=s["buffer"],
                                           workspace=s["workspace"], cap=s["cap"], slopes=s["slope"],
                                           window=s["window"], first=s["first"], last=s["last"])
    s["meta"].copy_(s["before"])
    if s["op"] == "branch":
        pisa.cache_fork(s["pool"], s["parents"], s["lengths"], workspace=s["workspace"])
        pisa.cache_reserve(s["pool"], s["lengths"], s["T"], granted=s["granted"], workspace=s["workspace"])
        return s["table"], s["refs"], s["lengths"], s["granted"], s["pages"]
    pisa.cache_compact(s["pool"], used=s["used"], workspace=s["workspace"])
    return s["table"], s["refs"], s["used"], s["pages"]


def run(s):
    if own:
        return _own(s)
    return {"append": _plain_append, "token": _plain_token, "prompt": _plain_prompt, "branch": _plain_branch,
            "compact": _plain_compact}[s["op"]](s)


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


def _exact_append(s):
    dev, half = s["q"].device, s["rot"] // 2
    q_out, k_out = s["q_out"].double(), s["k_out"].double()
    pages = s["pages"].double() if s["kind"] == "bf16" else None
    k_read, v_read = torch.zeros_like(k_out), torch.zeros_like(k_out)
    U = min(s["page"], 64)
    i = torch.arange(half, device=dev)
    a, b2 = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)

    def turn(x, cos, sin):
        y = x.double().clone()
        y[..., a] = x[..., a].double() * cos - x[..., b2].double() * sin
        y[..., b2] = x[..., a].double() * sin + x[..., b2].double() * cos
        return y

    for b in range(s["B"]):
        m = int(s["counts"][b])
        pos = int(s["start"][b]) + torch.arange(m, device=dev)
        cos = torch.empty(m, 1, half, dtype=torch.float64, device=dev)
        sin = torch.empty_like(cos)
        for pair, axis in enumerate(s["axes"]):
            p = s["positions"][axis, b, :m].long()
            cos[:, 0, pair], sin[:, 0, pair] = s["rotary"][p, pair].double(), s["rotary"][p, half + pair].double()
        q_out[b, :m] = turn(s["q"][b, :m], cos, sin)
        k = turn(s["k"][b, :m], cos, sin)
        k_out[b, :m] = k
        v = s["v"][b, :m].double()
        if pages is None:  # the cache holds what the keys are in bf16, in 4 bits
            k_read[b, :m], v_read[b, :m] = _exact_round(k.to(torch.bfloat16).double()), _exact_round(v)
        else:
            page, part, u = s["table"][b].long()[pos // s["page"]], pos % s["page"] // U, pos % U
            pages[page, :, part, 0, u], pages[page, :, part, 1, u] = k, v
    return (q_out, k_out, pages) if pages is not None else (q_out, k_out, k_read, v_read)


def _exact_attention(s):
    dev, T, G = s["q"].device, s["T"], s["Hq"] // s["Hkv"]
    out = torch.zeros(s["B"], T, s["Hq"], D, dtype=torch.float64, device=dev)
    for b in range(s["B"]):
        n = int(s["lengths"][b])
        m = T if s["op"] == "token" else int(s["counts"][b])
        p = n - m + torch.arange(m, device=dev)
        lo, hi = torch.zeros_like(p), p + 1
        if s["op"] == "prompt":
            lo = lo if s["first"] is None else s["first"][b, :m].long()
            hi = hi if s["last"] is None else s["last"][b, :m].long()
        if s["window"]:
            lo = torch.maximum(lo, p + 1 - s["window"])
        left = max(0, int(lo.min()))
        keys = torch.arange(left, n, device=dev)
        k, v = _exact_tokens(s, b, keys)
        step = max(1, (1 << 27) // (G * keys.numel()))
        for i in range(0, m, step):
            j = slice(i, min(i + step, m))
            hidden = (keys < lo[j, None]) | (keys >= hi[j, None])
            for h in range(s["Hkv"]):
                q = s["q"][b, j, h * G:(h + 1) * G].double()
                z = (q.reshape(-1, D) @ k[:, h].T).reshape(q.shape[0], G, -1) / 8
                if s["cap"]:
                    z = torch.tanh(z / s["cap"]) * s["cap"]
                if s["slope"] is not None:
                    z -= s["slope"][h * G:(h + 1) * G, None].double() * (p[j, None, None] - keys).abs()
                z.masked_fill_(hidden[:, None], -math.inf)
                w = torch.nan_to_num(torch.softmax(z, -1), nan=0.0)  # (a row that sees nothing)
                out[b, j, h * G:(h + 1) * G] = (w.flatten(0, 1) @ v[:, h]).reshape(q.shape)
    return out


def _exact_branch(s):
    P, n_pages, B = s["page"], s["n_pages"], s["B"]
    table, refs, lengths = s["table"].tolist(), s["refs"].tolist(), s["lengths"].tolist()
    rows, ns = [], []
    for q in s["parents"].tolist():
        rows.append(list(table[q]) if q >= 0 else [-1] * s["wide"])
        ns.append(lengths[q] if q >= 0 else 0)
    for x in sum(table, []):
        refs[x] -= x >= 0
    for x in sum(rows, []):
        refs[x] += x >= 0
    pages = s["pages"].double()
    before, free, granted, copies = list(refs), [x for x in range(n_pages) if refs[x] == 0], [], []
    taken = 0
    for b in range(B):
        first, stop = ns[b] // P, -(-(ns[b] + s["T"]) // P)
        want = [e for e in range(first, stop) if rows[b][e] < 0 or before[rows[b][e]] > 1] if stop <= s["wide"] else None
        if want is None or (want and taken + len(want) > len(free)):
            taken += len(want or [])
            granted.append(0)
            continue
        for e in want:
            x, y = rows[b][e], free[taken]
            taken += 1
            if x >= 0:
                refs[x] -= 1
                if e == first and ns[b] % P:
                    copies.append((x, y))
            refs[y] = 1
            rows[b][e] = y
        granted.append(s["T"])
    for x, y in copies:
        pages[y] = pages[x]
    return tuple(torch.tensor(z) for z in (rows, refs, ns, granted)) + (pages,)


def _exact_compact(s):
    table, refs = s["table"].tolist(), s["refs"].tolist()
    used = sum(x != 0 for x in refs)
    holes = [x for x in range(used) if refs[x] == 0]
    to = dict(zip([x for x in range(used, len(refs)) if refs[x]], holes))
    pages = s["pages"].double()
    for x, y in to.items():
        pages[y] = pages[x]
        refs[y], refs[x] = refs[x], 0
    return torch.tensor([[to.get(x, x) for x in row] for row in table]), torch.tensor(refs), torch.tensor([used]), pages


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "append":
        return _exact_append(s)
    if s["op"] in ("token", "prompt"):
        return _exact_attention(s)
    out = _exact_branch(s) if s["op"] == "branch" else _exact_compact(s)
    return tuple(x if x.is_floating_point() else x.to(torch.int32) for x in out)
