"""Measured cases of a decode step around a key/value cache held in 4 bits: the append that quantizes
to it, attention over it with an optional sliding window and first tokens that stay visible, the
norms before and after a block with its gate and residual scale, and a mixture-of-experts layer for
a few tokens on 4-bit experts.

Case fields: "op" picks the operator; "t" tokens, "b" sequences, "n" new tokens per sequence, "hq" /
"hkv" query and key/value heads, "d" head size, "group" elements that share a scale, "len" longest
sequence, "window" / "sinks" (window 0: all keys), "w" width of a row, "e" experts, "k" experts per
token, "h" hidden size, "i" an expert's inner size, "dtype" "fp16" or "bf16".

The cache is a uint8 tensor [pages, heads, page_size * (d + 8 * d / group)].  Tokens go in tiles of
16, a tile's bytes being: codes of the keys, codes of the values, (scale, minimum) of the keys' groups
as [token][group] pairs of 16-bit elements, the same of the values.  A code c stands for c * scale +
minimum.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
MAX_POSITION = 32768


def listed():
    return [
        # one user's chat in a serving loop: the call's latency counts
        {"name": "attention 1 over 700", "op": "attention", "b": 1, "n": 1, "hq": 32, "hkv": 8, "d": 128, "group": 128,
         "len": 700, "window": 0, "sinks": 0, "page": 16, "dtype": "fp16"},
        # a small batch under a sliding window whose first tokens stay visible, one key/value head per query head
        {"name": "attention 6 window 1024", "op": "attention", "b": 6, "n": 1, "hq": 40, "hkv": 40, "d": 96, "group": 32,
         "len": 9001, "window": 1024, "sinks": 4, "page": 32, "dtype": "bf16"},
        # several drafted tokens checked at once, small heads, finer groups
        {"name": "attention 16x4 over 2047", "op": "attention", "b": 16, "n": 4, "hq": 24, "hkv": 4, "d": 64, "group": 32,
         "len": 2047, "window": 0, "sinks": 0, "page": 48, "dtype": "fp16"},
        # a few very long documents
        {"name": "attention 4 over 131072", "op": "attention", "b": 4, "n": 1, "hq": 64, "hkv": 8, "d": 128, "group": 64,
         "len": 131072, "window": 0, "sinks": 0, "page": 64, "dtype": "bf16"},
        # a serving batch of a 70B-shaped layer, ragged
        {"name": "attention 128 over 8197", "op": "attention", "b": 128, "n": 1, "hq": 64, "hkv": 8, "d": 128, "group": 128,
         "len": 8197, "window": 0, "sinks": 0, "page": 16, "dtype": "bf16"},
        # one decode step of eight sequences
        {"name": "append 8 tokens", "op": "append", "t": 8, "hq": 64, "hkv": 8, "d": 128, "group": 128, "rot": 128,
         "interleaved": False, "page": 16, "dtype": "bf16"},
        # a prefill batch, rotated in part, pairs side by side
        {"name": "append 8191 tokens", "op": "append", "t": 8191, "hq": 32, "hkv": 8, "d": 128, "group": 64, "rot": 64,
         "interleaved": True, "page": 64, "dtype": "fp16"},
        # one decode step between attention and the experts: the residual sum and the next norm
        {"name": "norm 4 of 8192", "op": "norm", "t": 4, "w": 8192, "kind": "rms", "post": False, "gate": "none",
         "scale": 1.0, "dtype": "fp16"},
        # a prefill batch with a norm on either side of the sum, gate and residual scale
        {"name": "norm 8191 of 5120", "op": "norm", "t": 8191, "w": 5120, "kind": "rms", "post": True, "gate": "row",
         "scale": 0.25, "dtype": "bf16"},
        # one token of a small model's layer with many small experts
        {"name": "moe 1 token 8 of 128", "op": "moe", "t": 1, "e": 128, "k": 8, "h": 2048, "i": 768, "group": 128,
         "base": True, "dtype": "bf16"},
        # a few sequences, few large experts
        {"name": "moe 3 tokens 2 of 8", "op": "moe", "t": 3, "e": 8, "k": 2, "h": 4096, "i": 14336, "group": 128,
         "base": True, "dtype": "fp16"},
        # the largest batch of the form for a few tokens: most of the experts are read
        {"name": "moe 16 tokens 8 of 128", "op": "moe", "t": 16, "e": 128, "k": 8, "h": 4096, "i": 1792, "group": 128,
         "base": False, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "append", "norm", "norm", "moe", "moe"])
    dtype = rng.choice(["fp16", "bf16"])
    if op in ("attention", "append"):
        hkv, group_heads = rng.choice([(40, 1), (8, 8), (8, 5), (4, 7), (1, 16), (2, 7)])
        d, group = rng.choice([(64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (128, 128), (256, 64), (256, 128)])
        c = {"op": op, "hq": hkv * group_heads, "hkv": hkv, "d": d, "group": group, "page": rng.choice([16, 32, 48, 64, 128]),
             "dtype": dtype}
    if op == "attention":
        window = rng.choice([0, 0, 0, 1, 2])
        c.update({"b": _log(rng, 1, 128), "n": rng.choice([1, 1, 1, 2, 5]), "len": _log(rng, 1, 131072),
                  "window": _log(rng, 16, 8192) if window else 0, "sinks": rng.choice([1, 4, 100]) if window == 2 else 0})
        while c["b"] * c["len"] * hkv * d > 128 * 8197 * 8 * 128 or c["b"] * c["n"] * c["len"] * c["hq"] > 128 * 8197 * 64:
            c["b"], c["len"] = max(1, c["b"] // 2), c["len"] if c["b"] > 1 else c["len"] // 2
        return c
    if op == "append":
        c.update({"t": _log(rng, 1, 8191), "rot": rng.choice([d, d, d // 2]), "interleaved": rng.random() < 0.5})
        while c["t"] * (c["hq"] + 2 * hkv) * d > 8191 * 48 * 128:
            c["t"] = max(1, c["t"] // 2)
        return c
    if op == "norm":
        c = {"op": op, "t": _log(rng, 1, 8191), "w": rng.choice([512, 1000, 2048, 2880, 4096, 5120, 7168, 8192, 16384]),
             "kind": rng.choice(["rms", "rms", "layer"]), "post": rng.random() < 0.5, "gate": rng.choice(["none", "channel", "row"]),
             "scale": rng.choice([1.0, 0.25, 1.4]), "dtype": dtype}
        while c["t"] * c["w"] > 8191 * 5120:
            c["t"] = max(1, c["t"] // 2)
        return c
    e, k, h, i = rng.choice([(8, 2, 1024, 512), (8, 2, 4096, 14336), (64, 6, 2048, 1408), (60, 4, 2048, 1408), (128, 8, 2048, 768),
                             (128, 8, 4096, 1792), (256, 8, 7168, 2048)])
    t = _log(rng, 1, 16)
    while _distinct(t, k, e) * h * i > _distinct(16, 8, 128) * 4096 * 1792:
        t = max(1, t // 2)
    return {"op": op, "t": t, "e": e, "k": k, "h": h, "i": i, "group": rng.choice([128, 128, 64]) if i % 128 == 0 else 64,
            "base": rng.random() < 0.5, "dtype": dtype}


def _distinct(t, k, e):
    """Experts that t tokens of k of e experts are expected to need."""
    return e * (1.0 - (1.0 - k / e) ** t)


# ------------------------------------------------------------------------------ 4-bit cells ----

def _quantize(x, group):
    """Codes uint8, scale and minimum of the groups of the last dimension."""
    by = x.float().unflatten(-1, (-1, group))
    low = by.amin(-1, keepdim=True)
    scale = ((by.amax(-1, keepdim=True) - low) / 15.0).to(x.dtype)
    codes = torch.where(scale > 0, torch.round((by - low) / scale.float()).clamp(0, 15), 0.0)
    return codes.to(torch.uint8).flatten(-2), scale[..., 0], low[..., 0].to(x.dtype)


def _values(codes, scale, low):
    """What the codes stand for, in 32 bits."""
    by = codes.unflatten(-1, (scale.shape[-1], -1)).float()
    return (by * scale.float()[..., None] + low.float()[..., None]).flatten(-2)


def _key_bytes(codes):
    """Codes of keys [..., tokens, d] as the tiles' bytes [..., tiles, 8 d]."""
    d = codes.shape[-1]
    pairs = codes[..., 0::2] | codes[..., 1::2] << 4
    panels = max(1, d // 128)
    by = pairs.unflatten(-1, (panels, d // panels // 32, 4, 4)).unflatten(-5, (-1, 16))  # tile, token, panel, w, t, byte
    return by.movedim(-4, -5).transpose(-2, -3).flatten(-5)


def _key_codes(data, d):
    panels = max(1, d // 128)
    by = data.unflatten(-1, (panels, 16, 4, d // panels // 32, 4)).transpose(-2, -3).movedim(-5, -4).flatten(-4)
    return torch.stack([by & 15, by >> 4], dim=-1).flatten(-2).flatten(-3, -2)


def _value_bytes(codes):
    """Codes of values [..., tokens, d] as the tiles' bytes [..., tiles, 8 d]."""
    pairs = codes[..., 0::2] | codes[..., 1::2] << 4
    by = pairs.unflatten(-1, (-1, 8, 2)).unflatten(-4, (-1, 2, 4, 2))  # tile, half, t, odd, u, g, byte
    full = by.shape[-3] // 2 * 2
    both = by[..., :full, :, :].unflatten(-3, (-1, 2))  # tile, half, t, odd, pair, of the pair, g, byte
    both = both.movedim((-4, -2, -6, -3, -7, -5), (-7, -6, -5, -4, -3, -2)).flatten(-7)
    last = by[..., full:, :, :].movedim((-3, -2, -5, -6, -4), (-6, -5, -4, -3, -2)).flatten(-6)
    return torch.cat([both, last], dim=-1)


def _value_codes(data, d):
    full = d // 64 * 512
    both = data[..., :full].unflatten(-1, (-1, 8, 4, 2, 2, 2, 2))  # pair, g, t, of the pair, half, odd, byte
    both = both.movedim((-3, -5, -2, -7, -4, -6), (-7, -6, -5, -4, -3, -2)).flatten(-4, -3)
    last = data[..., full:].unflatten(-1, (-1, 8, 4, 2, 2, 2))  # u, g, t, half, odd, byte
    last = last.movedim((-3, -4, -2, -6, -5), (-6, -5, -4, -3, -2))
    by = torch.cat([both, last], dim=-3).flatten(-3)  # tile, half, t, odd, d / 2
    return torch.stack([by & 15, by >> 4], dim=-1).flatten(-2).flatten(-5, -2)


def _pack(k, v, group):
    """The cache of keys and values [pages, page_size, heads, d]."""
    parts = []
    for x, to_bytes in ((k, _key_bytes), (v, _value_bytes)):
        codes, scale, low = _quantize(x.transpose(1, 2), group)
        pairs = torch.stack([scale, low], dim=-1).unflatten(2, (-1, 16)).flatten(3).view(torch.uint8)
        parts.append((to_bytes(codes), pairs))
    (kc, kp), (vc, vp) = parts
    return torch.cat([kc, vc, kp, vp], dim=-1).flatten(2)


def _unpack(cache, d, group, dtype):
    """Keys and values [..., tokens, d] in 32 bits of cells [..., bytes]."""
    groups = d // group
    tiles = cache.unflatten(-1, (-1, 16 * (d + 8 * groups)))
    kc, vc, kp, vp = tiles.split([8 * d, 8 * d, 64 * groups, 64 * groups], dim=-1)
    params = [p.contiguous().view(dtype).unflatten(-1, (16, groups, 2)).flatten(-4, -3) for p in (kp, vp)]
    return (_values(codes, p[..., 0], p[..., 1]) for codes, p in zip((_key_codes(kc, d), _value_codes(vc, d)), params))


def _places(to_bytes, d):
    """Byte of a tile's codes where token r's elements 2 i, 2 i + 1 stand, [16, d / 2]."""
    pair = torch.arange(8 * d, device="cuda").view(16, d // 2)
    held = torch.zeros((8 * d,), dtype=torch.int64, device="cuda")
    for shift in (0, 4, 8, 12):  # the numbers of the pairs go through the layout four bits at a time, as codes
        part = pair >> shift & 15
        held += (to_bytes(torch.stack([part, part], dim=-1).flatten(1).to(torch.uint8)).flatten() & 15).long() << shift
    return torch.empty_like(held).scatter_(0, held, torch.arange(8 * d, device="cuda")).view(16, d // 2)


# ---------------------------------------------------------------------------------- inputs ----

def _lens(c):
    """Lengths, ragged; the same ones for every seed, in another order.  A batch of several has a slot
    without a sequence."""
    b, n, top = c["b"], c["n"], c["len"]
    lens = [min(top, n + (max(0, top - n) * (2 * i + 2 + b)) // (3 * b)) for i in range(b)]
    if b > 4:
        lens[0] = 0
    return lens


def _prepare_attention(c, g):
    dt, b, n, hq, hkv, d, page = DTYPES[c["dtype"]], c["b"], c["n"], c["hq"], c["hkv"], c["d"], c["page"]
    lens = torch.tensor(_lens(c), device="cuda", dtype=torch.int64)[torch.randperm(b, generator=g, device="cuda")]
    per = -(-c["len"] // page)
    total = b * per + 1
    pages = torch.randperm(total, generator=g, device="cuda")[:b * per].view(b, per)
    cache = torch.empty((total, hkv, page * (d + 8 * d // c["group"])), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (page * hkv * d))
    for first in range(0, total, step):
        count = min(step, total - first)
        # some channels of the keys are far from zero
        shift = 2.0 * torch.randn((hkv, d), generator=g, device="cuda") * (torch.rand((hkv, d), generator=g, device="cuda") < 0.1)
        k = (torch.randn((count, page, hkv, d), generator=g, device="cuda") + shift).to(dt)
        v = torch.randn((count, page, hkv, d), generator=g, device="cuda").to(dt)
        cache[first:first + count] = _pack(k, v, c["group"])
    # what no token was written to is never read: its scales and minima are NaN
    live = torch.zeros((total, page), dtype=torch.bool, device="cuda")
    live[pages.reshape(-1)] = (torch.arange(per * page, device="cuda")[None] < lens[:, None]).view(b * per, page)
    params = cache.view(total, hkv, page // 16, -1)[..., 16 * d:].unflatten(-1, (2, 16, -1))
    params.masked_fill_(~live.view(total, 1, page // 16, 1, 16, 1), 255)
    # queries that single some keys out
    q = (2.0 * torch.randn((b, n, hq, d), generator=g, device="cuda")).to(dt)
    return {"q": q, "cache": cache, "pages": pages.to(torch.int32).contiguous(), "lens": lens.to(torch.int32), "group": c["group"],
            "window": c["window"], "sinks": c["sinks"], "scale": 1.0 / math.sqrt(d)}


def _turn(x, cos, sin, interleaved):
    """x with its first elements rotated, products and sums rounded one by one in x's type."""
    rot = 2 * cos.shape[-1]
    turn, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
    else:
        a, b = turn[..., :rot // 2], turn[..., rot // 2:]
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], dim=-1).flatten(-2) if interleaved else torch.cat([u, v], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _clear(k, cos, sin, interleaved, dt):
    """Pairs whose rotated elements do not hang on the last bits of 32-bit products, per element of k."""
    x, cos, sin = k.double(), cos.double(), sin.double()
    turned, size = _turn(x, cos, sin, interleaved), _turn(x.abs(), cos.abs(), -sin.abs(), interleaved)
    # b cos + a sin has a sign of its own: the sum of both sizes bounds either
    size = torch.maximum(size.abs(), _turn(x.abs(), cos.abs(), sin.abs(), interleaved).abs())
    ok = (turned - 2.0 ** -22 * size).to(dt) == (turned + 2.0 ** -22 * size).to(dt)
    rot = 2 * cos.shape[-1]
    pair = ok[..., :rot].unflatten(-1, (rot // 2, 2) if interleaved else (2, rot // 2))
    both = pair.all(-1 if interleaved else -2, keepdim=True).expand_as(pair).flatten(-2)
    return torch.cat([both, torch.ones_like(ok[..., rot:])], dim=-1)


def _prepare_append(c, g):
    dt, t, hq, hkv, d, page = DTYPES[c["dtype"]], c["t"], c["hq"], c["hkv"], c["d"], c["page"]
    half = c["rot"] // 2
    angle = torch.arange(MAX_POSITION, dtype=torch.float64, device="cuda")[:, None] \
        * 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    table = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    positions = torch.randint(0, MAX_POSITION, (t,), generator=g, device="cuda", dtype=torch.int32)
    qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=g, device="cuda").to(dt)  # the fused linear's rows
    k = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
    line = table[positions.long()][:, None]
    # A rotated key whose rounding hangs on the last bits of 32-bit sums has no one right code: such
    # pairs are drawn again, and zero where that did not help.
    for again in (1.0, 1.0, 0.0):
        fresh = again * torch.randn(k.shape, generator=g, device="cuda")
        k.copy_(torch.where(_clear(k, line[..., :half], line[..., half:], c["interleaved"], dt), k, fresh.to(dt)))
    pages = -(-2 * t // page) + 1
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:t].to(torch.int32)
    if t > 1000:  # a prefill: runs of tokens in pages of their own
        order = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(t, device="cuda")
        slots = (order[at // page] * page + at % page).to(torch.int32)
    return {"q": qkv[:, :hq * d].view(t, hq, d), "k": k, "v": qkv[:, (hq + hkv) * d:].view(t, hkv, d), "positions": positions,
            "table": table, "interleaved": c["interleaved"], "group": c["group"], "slots": slots,
            "places": [_places(to_bytes, d) for to_bytes in (_key_bytes, _value_bytes)],
            "cache": torch.zeros((pages, hkv, page * (d + 8 * d // c["group"])), dtype=torch.uint8, device="cuda")}


def _prepare_norm(c, g):
    dt, t, w = DTYPES[c["dtype"]], c["t"], c["w"]
    draw_ = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = {"x": (3.0 * draw_(t, w) + 0.5).to(dt), "residual": (10.0 * draw_(t, w)).to(dt), "weight": (1.0 + 0.1 * draw_(w)).to(dt),
         "kind": c["kind"], "scale": c["scale"], "eps": 1e-6, "post_weight": (1.0 + 0.1 * draw_(w)).to(dt) if c["post"] else None}
    layer = c["kind"] == "layer"
    s["bias"] = (0.1 * draw_(w)).to(dt) if layer else None
    s["post_bias"] = (0.1 * draw_(w)).to(dt) if layer and c["post"] else None
    s["gate"] = None if c["gate"] == "none" else draw_(*((w,) if c["gate"] == "channel" else (t, w))).to(dt)
    return s


def _weights(g, e, k, n, group, dt):
    """Stacked 4-bit linears [e, k, n] whose outputs keep the size of their inputs."""
    word = lambda *shape: torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)  # noqa: E731
    scales = (torch.rand((e, k // group, n), generator=g, device="cuda") * 0.2 + 0.05) / math.sqrt(k)
    return [word(e, k, n // 8), word(e, k // group, n // 8), scales.to(dt)]


def _prepare_moe(c, g):
    dt, t, e, k = DTYPES[c["dtype"]], c["t"], c["e"], c["k"]
    favour = 0.5 * torch.randn((e,), generator=g, device="cuda")
    experts = (favour + torch.randn((t, e), generator=g, device="cuda")).topk(k, dim=-1).indices.to(torch.int32)
    weights = torch.rand((t, k), generator=g, device="cuda") + 0.05
    return {"x": torch.randn((t, c["h"]), generator=g, device="cuda").to(dt), "experts": experts,
            "weights": weights / weights.sum(-1, keepdim=True), "group": c["group"],
            "up": _weights(g, e, c["h"], 2 * c["i"], c["group"], dt), "down": _weights(g, e, c["i"], c["h"], c["group"], dt),
            "base": torch.randn((t, c["h"]), generator=g, device="cuda").to(dt) if c["base"] else None}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    make = {"attention": _prepare_attention, "append": _prepare_append, "norm": _prepare_norm, "moe": _prepare_moe}[case["op"]]
    return {"op": case["op"], **make(case, g)}


# ------------------------------------------------------------------------------ plain forms ----

def _plain_attention(s):
    b, n, hq, d = s["q"].shape
    hkv = s["cache"].shape[1]
    cells = s["cache"][s["pages"].long()].transpose(1, 2).flatten(2, 3)  # [b, hkv, bytes]
    k, v = _unpack(cells, d, s["group"], s["q"].dtype)
    q = s["q"].float().view(b, n, hkv, -1, d).permute(0, 2, 1, 3, 4).flatten(2, 3) * s["scale"]
    j = torch.arange(k.shape[2], device=q.device)
    at = (s["lens"][:, None] - n + torch.arange(n, device=q.device))[..., None]  # positions of the new tokens
    seen = j <= at
    if s["window"]:
        seen &= (j > at - s["window"]) | (j < s["sinks"])
    seen = seen[:, None, :, None].expand(-1, hkv, -1, hq // hkv, -1).flatten(2, 3)
    live = j[None] < s["lens"][:, None]
    k, v = (x.masked_fill(~live[:, None, :, None], 0.0) for x in (k, v))
    z = torch.where(seen, q @ k.transpose(2, 3), float("-inf"))
    p = torch.where(seen, torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-3e38)), 0.0)
    out = (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return out.view(b, hkv, n, -1, d).permute(0, 2, 1, 3, 4).reshape(b, n, hq, d).to(s["q"].dtype)


def _plain_append(s):
    dt, (t, hkv, d), group = s["q"].dtype, s["k"].shape, s["group"]
    line = s["table"][s["positions"].long()][:, None]
    half = line.shape[-1] // 2
    cos, sin = line[..., :half], line[..., half:]
    q = _turn(s["q"].float(), cos, sin, s["interleaved"]).to(dt)
    k = _turn(s["k"].float(), cos, sin, s["interleaved"]).to(dt)
    groups = d // group
    tiles = s["cache"].view(*s["cache"].shape[:2], -1, 16 * (d + 8 * groups))
    slot = s["slots"].long()
    page, at, row = slot // (16 * tiles.shape[2]), slot // 16 % tiles.shape[2], slot % 16
    out = [q]
    for x, first in ((k, 0), (s["v"], 1)):
        codes, scale, low = _quantize(x, group)
        out.append(_values(codes, scale, low).to(dt))
        place = s["places"][first][row] + first * 8 * d  # [t, d / 2]
        pairs = codes[..., 0::2] | codes[..., 1::2] << 4
        heads = torch.arange(hkv, device=x.device)[None, :, None]
        tiles[page[:, None, None], heads, at[:, None, None], place[:, None]] = pairs
        params = torch.stack([scale, low], dim=-1).flatten(2).view(torch.uint8)
        place = 16 * d + first * 64 * groups + row[:, None] * 4 * groups + torch.arange(4 * groups, device=x.device)
        tiles[page[:, None, None], heads, at[:, None, None], place[:, None]] = params
    return out


def _norm(x, kind, eps):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)


def _plain_norm(s):
    x = s["x"].float()
    if s["post_weight"] is not None:
        x = _norm(x, s["kind"], s["eps"]) * s["post_weight"].float()
        if s["post_bias"] is not None:
            x = x + s["post_bias"].float()
    if s["gate"] is not None:
        x = x * s["gate"].float()
    h = s["residual"].float() + s["scale"] * x
    y = _norm(h, s["kind"], s["eps"]) * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return [h.to(s["x"].dtype), y.to(s["x"].dtype)]


ORDER = (0, 2, 4, 6, 1, 3, 5, 7)  # nibble i of a word holds the column ORDER[i] of its eight


def _nibbles(words):
    shifts = torch.tensor([4 * ORDER.index(j) for j in range(8)], device=words.device, dtype=torch.int32)
    return (words[..., None] >> shifts & 15).flatten(-2)


def _dequantized(linear, ids, group):
    """Weights [places, k, n] in 32 bits of the experts `ids`."""
    qweight, qzeros, scales = (x[ids] for x in linear)
    codes = _nibbles(qweight).float().unflatten(1, (-1, group))
    return ((codes - _nibbles(qzeros).float()[:, :, None]) * scales.float()[:, :, None]).flatten(1, 2)


def _plain_moe(s):
    t, k = s["experts"].shape
    ids = s["experts"].flatten().long()
    x = s["x"].float().repeat_interleave(k, dim=0)[:, None]  # [places, 1, h]
    gate, up = (x @ _dequantized(s["up"], ids, s["group"])).chunk(2, dim=-1)
    act = gate / (1.0 + torch.exp(-gate)) * up
    y = (act @ _dequantized(s["down"], ids, s["group"])).view(t, k, -1)
    y = (y * s["weights"][..., None]).sum(1)
    if s["base"] is not None:
        y = y + s["base"].float()
    return y.to(s["x"].dtype)


def _own(s):
    import w4a16_weight_only_gb300 as awq
    op = s["op"]
    if op == "attention":
        return awq.awq_attention_kv4(s["q"], s["cache"], s["pages"], s["lens"], group_size=s["group"], window=s["window"],
                                     sinks=s["sinks"], scale=s["scale"])
    if op == "append":
        q = awq.awq_rope_append_kv4(s["q"], s["k"], s["v"], s["positions"], s["table"], s["cache"], s["slots"],
                                    group_size=s["group"], interleaved=s["interleaved"])
        k, v = awq.awq_kv4_read(s["cache"], s["slots"], s["k"].shape[2], group_size=s["group"], dtype=s["k"].dtype)
        return [q, k, v]
    if op == "norm":
        return list(awq.awq_residual_norm(s["x"], s["residual"], weight=s["weight"], bias=s["bias"], post_weight=s["post_weight"],
                                          post_bias=s["post_bias"], gate=s["gate"], scale=s["scale"], eps=s["eps"],
                                          kind=s["kind"]))
    return awq.awq_moe_layer(s["x"], s["weights"], s["experts"], s["up"], s["down"], group_size=s["group"], base=s["base"])


def run(state):
    if own:
        return _own(state)
    return {"attention": _plain_attention, "append": _plain_append, "norm": _plain_norm, "moe": _plain_moe}[state["op"]](state)


# ------------------------------------------------------------------------------------ work ----

def _seen(c, length):
    """Keys that the new tokens of a sequence see: of any of them, and summed over them."""
    n, window, sinks = c["n"], c["window"], c["sinks"]
    total, lowest = 0, length
    for at in range(max(0, length - n), length):
        first = max(0, at - window + 1) if window else 0
        total += at + 1 - first + min(first, sinks)
        lowest = min(lowest, first)
    return (length - lowest + min(lowest, sinks), total) if total else (0, 0)


def work(case):
    c, size = case, 2
    if c["op"] == "attention":
        seen = [_seen(c, x) for x in _lens(c)]
        cell = c["hkv"] * (c["d"] + 8 * c["d"] // c["group"])
        keys, pairs = sum(x for x, _ in seen), sum(x for _, x in seen)
        return {"bytes": keys * cell + 2 * c["b"] * c["n"] * c["hq"] * c["d"] * size + 4 * keys // c["page"] + 4 * c["b"],
                "flops": 4 * pairs * c["hq"] * c["d"]}
    if c["op"] == "append":  # the append, and the read of the same cells
        cell = c["hkv"] * (c["d"] + 8 * c["d"] // c["group"])
        rows = 2 * (c["hq"] + 2 * c["hkv"]) * c["d"] * size
        return {"bytes": c["t"] * (rows + 2 * cell + 4 * c["rot"] + 12), "flops": 3 * c["t"] * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] == "norm":
        rows = 4 + (1 if c["gate"] == "row" else 0)
        return {"bytes": (c["t"] * rows + 2) * c["w"] * size, "flops": c["t"] * c["w"] * (10 if c["post"] else 7)}
    weights = 3 * c["h"] * c["i"] * (0.5 + (size + 0.5) / c["group"])
    return {"bytes": int(_distinct(c["t"], c["k"], c["e"]) * weights) + c["t"] * c["h"] * size * (3 if c["base"] else 2),
            "flops": 6 * c["t"] * c["k"] * c["h"] * c["i"]}


# ----------------------------------------------------------------------------------- exact ----

def _cells64(s, pages, count, d):
    """Keys and values [count, heads, d] of the first tokens of the pages, by the address of each code."""
    groups, heads = d // s["group"], s["cache"].shape[1]
    tile_bytes = 16 * (d + 8 * groups)
    tiles = s["cache"].view(s["cache"].shape[0], heads, -1, tile_bytes)[pages].transpose(1, 2).flatten(0, 1)  # [tiles, heads, bytes]
    tiles = tiles[:-(-count // 16)]
    r, x = torch.arange(16, device="cuda")[:, None], torch.arange(d, device="cuda")[None]
    # keys: words of eight elements, those of a 128-element panel transposed four by four
    words = min(d, 128) // 32
    in_panel = x % 128 // 8
    k_at = x // 128 * 1024 + r * 16 * words + (in_panel % 4 * words + in_panel // 4) * 4 + x % 8 // 2
    # values: 16 tokens by 32 elements as two tokens by four elements in a word
    u, g, e = x // 32, x // 4 % 8, x // 2 % 2
    lane, inside = 4 * g + r // 2 % 4, r // 8 * 4 + r % 2 * 2 + e
    paired = u < d // 64 * 2
    v_at = 8 * d + torch.where(paired, u // 2 * 512 + lane * 16 + u % 2 * 8, d // 64 * 512 + lane * 8) + inside
    out = []
    for address, first in ((k_at, 0), (v_at, 1)):
        code = (tiles[:, :, address] >> (4 * (x % 2)) & 15).double()  # [tiles, heads, 16, d]
        p = tiles[:, :, 16 * d + first * 64 * groups:][:, :, :64 * groups].contiguous().view(s["q"].dtype)
        p = p.view(*p.shape[:2], 16, groups, 2).double().repeat_interleave(s["group"], dim=3)
        out.append((code * p[..., 0] + p[..., 1]).transpose(1, 2).flatten(0, 1)[:count])
    return out


def _exact_attention(c, s):
    hkv, n, rows = c["hkv"], c["n"], []
    for i, count in enumerate(s["lens"].tolist()):
        out = torch.zeros((n, hkv, c["hq"] // hkv, c["d"]), dtype=torch.float64, device="cuda")
        if count:
            k, v = _cells64(s, s["pages"][i, :-(-count // c["page"])].long(), count, c["d"])
            for a in range(n):
                at = count - n + a
                if at < 0:
                    continue
                keys = torch.arange(at + 1, device="cuda")
                if c["window"]:
                    keys = keys[(keys >= at - c["window"] + 1) | (keys < c["sinks"])]
                q = s["q"][i, a].double().view(hkv, -1, c["d"])
                p = torch.softmax(torch.einsum("hgd,jhd->hgj", q, k[keys]) / math.sqrt(c["d"]), dim=-1)
                out[a] = torch.einsum("hgj,jhd->hgd", p, v[keys])
        rows.append(out.reshape(n, c["hq"], c["d"]))
    return torch.stack(rows)


def _exact_append(c, s):
    half, dt = c["rot"] // 2, s["q"].dtype
    line = s["table"][s["positions"].long()].double()[:, None]
    turn = torch.complex(line[..., :half], line[..., half:])
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c["interleaved"] else (slice(0, half), slice(half, 2 * half))
    out = []
    for name in ("q", "k"):
        x = s[name].double().clone()
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        out.append(x)
    for x in (out.pop().to(dt), s["v"]):  # cells take the elements as a 16-bit cache would hold them
        by = x.double().view(c["t"], c["hkv"], -1, c["group"])
        low, high = by.min(-1, keepdim=True).values, by.max(-1, keepdim=True).values
        scale = ((high - low) / 15).to(dt).double()
        code = torch.round((by - low) / scale.clamp(min=1e-300)).clamp(0, 15)
        out.append((torch.where(scale > 0, code, 0.0) * scale + low).view(x.shape))
    return out


def _exact_norm(c, s):
    def norm(x):
        centred = x - x.mean(-1, keepdim=True) if c["kind"] == "layer" else x
        return centred / torch.sqrt(centred.square().mean(-1, keepdim=True) + s["eps"])

    x = s["x"].double()
    if c["post"]:
        x = norm(x) * s["post_weight"].double() + (s["post_bias"].double() if s["post_bias"] is not None else 0.0)
    if s["gate"] is not None:
        x = s["gate"].double() * x
    h = s["residual"].double() + c["scale"] * x
    return [h, norm(h) * s["weight"].double() + (s["bias"].double() if s["bias"] is not None else 0.0)]


def _exact_moe(c, s):
    def times(x, linear, e):
        qweight, qzeros, scales = (t[e] for t in linear)
        out = torch.empty((x.shape[0], scales.shape[1]), dtype=torch.float64, device="cuda")
        for i, column in enumerate(ORDER):
            w = (qweight >> 4 * i & 15).double().view(-1, c["group"], qweight.shape[1])
            z = (qzeros >> 4 * i & 15).double()[:, None]
            out[:, column::8] = x @ ((w - z) * scales[:, column::8].double()[:, None]).flatten(0, 1)
        return out

    out = s["base"].double() if s["base"] is not None else torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    for e in sorted(set(s["experts"].flatten().tolist())):
        token, place = (s["experts"] == e).nonzero(as_tuple=True)
        both = times(s["x"][token].double(), s["up"], e)
        gate, up = both[:, :c["i"]], both[:, c["i"]:]
        y = times(gate * torch.sigmoid(gate) * up, s["down"], e)
        out = out.index_add(0, token, y * s["weights"][token, place].double()[:, None])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "append": _exact_append, "norm": _exact_norm, "moe": _exact_moe}[case["op"]](case, s)
