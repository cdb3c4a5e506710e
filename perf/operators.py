"""Measured cases of the operators between a decoder layer's 4-bit linears: rotary positions (with
the append to a paged key/value cache), attention of a batch that shares a prefix, routing to
experts, and the dispatch / combine pair around the experts' grouped products.

Case fields: "op" picks the operator; "t" tokens, "b" sequences, "n" query tokens per sequence,
"hq" / "hkv" query and key/value heads, "d" head size, "rot" rotated part of the head, "e" experts,
"k" experts per token, "w" width of a row, "dtype" "fp16" or "bf16".
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4}


def listed():
    return [
        # one decode step of eight sequences: fused qkv rows in, keys and values into the cache
        {"name": "rope append 8 tokens", "op": "rope_append", "t": 8, "hq": 64, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "page": 16, "scaling": "none", "dtype": "bf16"},
        # a prefill chunk of a 7B-shaped layer whose heads are rotated in part, pairs side by side,
        # with positions scaled for a longer context
        {"name": "rope prefill 8191 tokens", "op": "rope", "t": 8191, "hq": 32, "hkv": 32, "d": 128, "rot": 64,
         "interleaved": True, "page": 0, "scaling": "yarn", "dtype": "fp16"},
        # a few short chats over one system prompt, one key/value head per query head
        {"name": "attention 3 over 1000", "op": "attention", "b": 3, "n": 1, "hq": 32, "hkv": 32, "d": 128,
         "prefix": 1000, "private": 100, "page": 16, "dtype": "bf16"},
        # several drafted tokens checked at once, small heads, pages that are no power of two
        {"name": "attention 16x4 over 2047", "op": "attention", "b": 16, "n": 4, "hq": 24, "hkv": 4, "d": 64,
         "prefix": 2047, "private": 700, "page": 20, "dtype": "fp16"},
        # a serving batch of a 70B-shaped layer
        {"name": "attention 64 over 8197", "op": "attention", "b": 64, "n": 1, "hq": 64, "hkv": 8, "d": 128,
         "prefix": 8197, "private": 1024, "page": 16, "dtype": "fp16"},
        # the same layer at its largest: many answers drawn from one long document
        {"name": "attention 128 over 32768", "op": "attention", "b": 128, "n": 1, "hq": 64, "hkv": 8, "d": 128,
         "prefix": 32768, "private": 2048, "page": 64, "dtype": "bf16"},
        # one decode step, two of eight experts
        {"name": "route 4 of 8", "op": "route", "t": 4, "e": 8, "k": 2, "scoring": "softmax", "bias": False,
         "groups": 1, "topk_groups": 1, "group_best": 1, "dtype": "fp16"},
        # a large prefill batch over many experts, limited to half of the groups
        {"name": "route 16381 of 256", "op": "route", "t": 16381, "e": 256, "k": 8, "scoring": "sigmoid", "bias": True,
         "groups": 8, "topk_groups": 4, "group_best": 2, "dtype": "fp32"},
        # one decode step of a small batch
        {"name": "dispatch 13 to 8", "op": "dispatch", "t": 13, "e": 8, "k": 2, "w": 4096, "dropped": 0.0, "dtype": "fp16"},
        # a prefill batch, some of its places without an expert (padding)
        {"name": "dispatch 8192 to 128", "op": "dispatch", "t": 8192, "e": 128, "k": 8, "w": 4096, "dropped": 0.05,
         "dtype": "bf16"},
        {"name": "combine 13", "op": "combine", "t": 13, "e": 8, "k": 2, "w": 4096, "dropped": 0.0, "base": True,
         "dtype": "fp16"},
        {"name": "combine 8192", "op": "combine", "t": 8192, "e": 128, "k": 8, "w": 4096, "dropped": 0.05, "base": False,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_append", "rope", "attention", "attention", "attention", "route", "dispatch", "combine"])
    dtype = rng.choice(["fp16", "bf16"])
    if op in ("rope", "rope_append"):
        hkv, group = rng.choice([(32, 1), (8, 8), (8, 4), (4, 6), (1, 16), (2, 7)])
        d = rng.choice([64, 96, 128, 256])
        c = {"op": op, "t": _log(rng, 1, 8191), "hq": hkv * group, "hkv": hkv, "d": d, "rot": rng.choice([d, d, d // 2]),
             "interleaved": rng.random() < 0.5, "page": rng.choice([16, 20, 64]) if op == "rope_append" else 0,
             "scaling": rng.choice(["none", "linear", "yarn"]), "dtype": dtype}
        while c["t"] * (c["hq"] + 2 * c["hkv"]) * d > 8191 * 96 * 128:
            c["t"] = max(1, c["t"] // 2)
        return c
    if op == "attention":
        hkv, group = rng.choice([(32, 1), (8, 8), (8, 4), (4, 6), (1, 16), (2, 7), (1, 64)])
        c = {"op": op, "b": _log(rng, 1, 128), "n": rng.choice([1, 1, 1, 2, 5]), "hq": hkv * group, "hkv": hkv,
             "d": rng.choice([64, 96, 128, 128, 128, 256]), "prefix": _log(rng, 1, 32768), "private": _log(rng, 1, 2048),
             "page": rng.choice([16, 16, 20, 64, 128]), "dtype": dtype}
        while (c["n"] * c["b"] * c["hq"] * c["prefix"] * max(c["d"], 128) > 128 * 64 * 32768 * 128
               or c["b"] * c["private"] * hkv * max(c["d"], 128) > 128 * 2048 * 8 * 128):
            c["b"] = max(1, c["b"] // 2)
        return c
    if op == "route":
        e, k, groups, topk_groups = rng.choice([(8, 2, 1, 1), (60, 4, 1, 1), (64, 6, 1, 1), (128, 8, 1, 1), (160, 6, 8, 3),
                                                (256, 8, 8, 4), (384, 8, 1, 1)])
        return {"op": op, "t": _log(rng, 1, 16381), "e": e, "k": k, "scoring": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": groups, "topk_groups": topk_groups,
                "group_best": rng.choice([1, 2]) if groups > 1 else 1, "dtype": rng.choice(["fp16", "bf16", "fp32"])}
    e, k = rng.choice([(8, 2), (60, 4), (64, 6), (128, 8), (256, 8)])
    c = {"op": op, "t": _log(rng, 1, 8192), "e": e, "k": k, "w": rng.choice([2048, 2880, 4096, 5120, 8192]),
         "dropped": rng.choice([0.0, 0.05]), "dtype": dtype}
    while c["t"] * (k + 1) * c["w"] > 8192 * 9 * 4096:
        c["t"] = max(1, c["t"] // 2)
    if op == "combine":
        c["base"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------------- inputs ----

def _frequencies(rot, scaling):
    """Frequencies of the rotated pairs and the factor on cos and sin, in 64 bits."""
    pair = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = 10000.0 ** (-2.0 * pair / rot)
    if scaling == "linear":
        return f / 4.0, 1.0
    if scaling == "yarn":  # by wavelength: fast pairs kept, slow pairs divided by the factor, a ramp between
        factor, original, fast, slow = 8.0, 4096, 32.0, 1.0
        at = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
        low, high = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
        ramp = ((pair - low) / max(high - low, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _table(last, rot, scaling):
    f, factor = _frequencies(rot, scaling)
    angle = torch.arange(last, dtype=torch.float64, device="cuda")[:, None] * f[None]
    return (torch.cat([angle.cos(), angle.sin()], dim=1) * factor).float()


MAX_POSITION = 32768


def _prepare_rope(c, g):
    dt, t, hq, hkv, d = DTYPES[c["dtype"]], c["t"], c["hq"], c["hkv"], c["d"]
    qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=g, device="cuda").to(dt)  # the fused linear's rows
    s = {"q": qkv[:, :hq * d].view(t, hq, d), "k": qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d),
         "v": qkv[:, (hq + hkv) * d:].view(t, hkv, d), "table": _table(MAX_POSITION, c["rot"], c["scaling"]),
         "interleaved": c["interleaved"]}
    if c["op"] == "rope":  # one chunk of one sequence
        first = int(torch.randint(0, MAX_POSITION - t + 1, (1,), generator=g, device="cuda"))
        s["positions"] = torch.arange(first, first + t, device="cuda", dtype=torch.int32)
        return s
    s["positions"] = torch.randint(0, MAX_POSITION, (t,), generator=g, device="cuda", dtype=torch.int32)
    pages = -(-2 * t // c["page"]) + 1
    for name in ("k_cache", "v_cache"):
        s[name] = torch.randn((pages, c["page"], hkv, d), generator=g, device="cuda").to(dt)
    s["slots"] = torch.randperm(pages * c["page"], generator=g, device="cuda")[:t].to(torch.int32)
    if t > 4:
        s["slots"][t // 2] = -1  # a padding token: nothing of it is kept
    return s


def _lens(c):
    """Private lengths, ragged; the same ones for every seed, in another order."""
    b, n, top = c["b"], c["n"], c["private"]
    return [min(top, n + (max(0, top - n) * (2 * i + 1)) // (2 * b)) for i in range(b)]


def _prepare_attention(c, g):
    dt, b, n, hq, hkv, d, page = DTYPES[c["dtype"]], c["b"], c["n"], c["hq"], c["hkv"], c["d"], c["page"]
    lens = torch.tensor(_lens(c), device="cuda", dtype=torch.int64)[torch.randperm(b, generator=g, device="cuda")]
    per = -(-c["private"] // page)
    shared = -(-c["prefix"] // page)
    total = shared + b * per + 1
    order = torch.randperm(total, generator=g, device="cuda")
    prefix_pages, pages = order[:shared], order[shared:shared + b * per].view(b, per)
    at = torch.arange(per * page, device="cuda")
    live = torch.zeros((total, page), dtype=torch.bool, device="cuda")
    in_prefix = torch.arange(shared * page, device="cuda") < c["prefix"]
    live[prefix_pages] = in_prefix.view(shared, page)
    live[pages.reshape(-1)] = (at[None] < lens[:, None]).view(b * per, page)
    s = {"prefix_len": c["prefix"], "prefix_pages": prefix_pages.to(torch.int32), "pages": pages.to(torch.int32).contiguous(),
         "lens": lens.to(torch.int32), "max_len": c["private"], "scale": 1.0 / math.sqrt(d)}
    for name in ("k_cache", "v_cache"):  # what no token was written to is never read: it holds NaN
        x = torch.randn((total, page, hkv, d), generator=g, device="cuda", dtype=torch.float32).to(dt)
        x.masked_fill_(~live[:, :, None, None], float("nan"))
        s[name] = x
    s["q"] = (2.0 * torch.randn((b, n, hq, d), generator=g, device="cuda")).to(dt)
    return s


def _keys64(logits, bias, c):
    """Scores and selection keys of the routing in 64 bits; keys of experts outside the kept groups
    are -inf."""
    x = logits.double()
    score = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.softmax(x, dim=-1)
    key = score if bias is None else score + bias.double()
    spread = []
    if c["groups"] > 1:
        by = key.view(key.shape[0], c["groups"], -1)
        best = by.sort(dim=-1, descending=True).values[..., :c["group_best"]].sum(-1)
        ranked, order = best.sort(dim=-1, descending=True, stable=True)
        spread.append(ranked[:, c["topk_groups"] - 1:c["topk_groups"] + 1])
        kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, order[:, :c["topk_groups"]], True)
        key = by.masked_fill(~kept[..., None], float("-inf")).reshape(key.shape)
    spread.append(key.sort(dim=-1, descending=True).values[:, :c["k"] + 1])
    return score, key, spread


def _prepare_route(c, g):
    t, e = c["t"], c["e"]
    bias = 0.1 * torch.randn((e,), generator=g, device="cuda") if c["bias"] else None
    drawn = (1.5 * torch.randn((t + t // 2 + 64, e), generator=g, device="cuda")).to(DTYPES[c["dtype"]])
    # A token whose choice hangs on the last bits of 32-bit scores has no one right answer: such rows
    # are left out. Equal scores stay: ties go to the lowest index.
    clear = torch.ones((drawn.shape[0],), dtype=torch.bool, device="cuda")
    for ranked in _keys64(drawn, bias, c)[2]:
        gap = ranked[:, :-1] - ranked[:, 1:]
        clear &= ((gap == 0) | (gap > 1e-5 * ranked[:, :-1].abs()) | ranked[:, 1:].isinf()).all(-1)
    rows = clear.nonzero()[:t, 0]
    return {"logits": drawn[rows].contiguous(), "bias": bias, "k": c["k"], "scoring": c["scoring"], "groups": c["groups"],
            "topk_groups": c["topk_groups"], "group_best": c["group_best"], "scale": 2.5}


def _experts(c, g):
    """Distinct experts per token, popular ones more often, some places without an expert."""
    t, e, k = c["t"], c["e"], c["k"]
    favour = torch.randn((e,), generator=g, device="cuda")
    ids = (favour + torch.randn((t, e), generator=g, device="cuda")).topk(k, dim=-1).indices.to(torch.int32)
    if c["dropped"]:
        ids[torch.rand((t, k), generator=g, device="cuda") < c["dropped"]] = -1
    return ids


def _rows_of(ids, e):
    """Row of each (token, place) among the rows sorted by expert, -1 without one; and the offsets."""
    flat = ids.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < e), flat, torch.full_like(flat, e))
    order = flat.sort(stable=True).indices
    rows = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=order.device))
    offsets = torch.zeros((e + 1,), dtype=torch.int64, device=ids.device)
    offsets[1:] = (flat[:, None] == torch.arange(e, device=ids.device)).sum(0).cumsum(0)
    return torch.where(flat < e, rows, torch.full_like(rows, -1)).view(ids.shape), offsets, order


def _prepare_dispatch(c, g):
    return {"x": torch.randn((c["t"], c["w"]), generator=g, device="cuda").to(DTYPES[c["dtype"]]), "experts": _experts(c, g),
            "e": c["e"]}


def _prepare_combine(c, g):
    dt, t, k, w = DTYPES[c["dtype"]], c["t"], c["k"], c["w"]
    rows, _, _ = _rows_of(_experts(c, g), c["e"])
    weights = torch.rand((t, k), generator=g, device="cuda") + 0.05
    return {"y": torch.randn((t * k, w), generator=g, device="cuda").to(dt), "weights": weights / weights.sum(-1, keepdim=True),
            "rows": rows.to(torch.int32), "base": torch.randn((t, w), generator=g, device="cuda").to(dt) if c["base"] else None}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    make = {"rope": _prepare_rope, "rope_append": _prepare_rope, "attention": _prepare_attention, "route": _prepare_route,
            "dispatch": _prepare_dispatch, "combine": _prepare_combine}[case["op"]]
    return {"op": case["op"], **make(case, g)}


# ------------------------------------------------------------------------------ plain forms ----

def _rotate(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    x = x.float()
    turn, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
    else:
        a, b = turn[..., :rot // 2], turn[..., rot // 2:]
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], dim=-1).flatten(-2) if interleaved else torch.cat([u, v], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _plain_rope(s):
    line = s["table"][s["positions"].long()][:, None]
    half = line.shape[-1] // 2
    cos, sin = line[..., :half], line[..., half:]
    q = _rotate(s["q"], cos, sin, s["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"], cos, sin, s["interleaved"]).to(s["k"].dtype)
    if s["op"] == "rope":
        return [q, k]
    kept = s["slots"] >= 0
    slots = s["slots"][kept].long()
    s["k_cache"].view(-1, *k.shape[1:])[slots] = k[kept]
    s["v_cache"].view(-1, *k.shape[1:])[slots] = s["v"][kept]
    return [q, s["k_cache"], s["v_cache"]]


def _plain_attention(s):
    b, n, hq, d = s["q"].shape
    page, hkv = s["k_cache"].shape[1:3]
    group = hq // hkv
    flat = lambda x: x.view(-1, hkv, d)  # noqa: E731
    q = s["q"].float().view(b, n, hkv, group, d) * s["scale"]
    at = torch.arange(s["prefix_len"], device=q.device)
    at = s["prefix_pages"].long()[at // page] * page + at % page
    k, v = (flat(s[x])[at].float().transpose(0, 1) for x in ("k_cache", "v_cache"))  # [hkv, prefix, d]
    shared = (q.permute(2, 0, 1, 3, 4).reshape(hkv, -1, d) @ k.transpose(1, 2)).view(hkv, b, n, group, -1)
    shared = shared.permute(1, 0, 2, 3, 4)  # [b, hkv, n, group, prefix]
    j = torch.arange(s["max_len"], device=q.device)
    at = s["pages"].long()[:, j // page] * page + j % page
    live = j[None] < s["lens"][:, None]
    pk, pv = (torch.where(live[..., None, None], flat(s[x])[at].float(), 0.0).transpose(1, 2) for x in ("k_cache", "v_cache"))
    own_ = (q.permute(0, 2, 1, 3, 4).reshape(b, hkv, n * group, d) @ pk.transpose(2, 3)).view(b, hkv, n, group, -1)
    seen = j[None, None] <= s["lens"][:, None, None] - n + torch.arange(n, device=q.device)[None, :, None]  # [b, n, j]
    own_ = torch.where(seen[:, None, :, None], own_, float("-inf"))
    top = torch.maximum(shared.amax(-1), own_.amax(-1))[..., None]
    shared, own_ = torch.exp(shared - top), torch.exp(own_ - top)
    total = shared.sum(-1) + own_.sum(-1)
    out = (shared.permute(1, 0, 2, 3, 4).reshape(hkv, b * n * group, -1) @ v).view(hkv, b, n, group, d).permute(1, 0, 2, 3, 4)
    out = out + (own_.reshape(b, hkv, n * group, -1) @ pv).view(b, hkv, n, group, d)
    out = out / total[..., None]
    return out.permute(0, 2, 1, 3, 4).reshape(b, n, hq, d).to(s["q"].dtype)


def _plain_route(s):
    x = s["logits"].float()
    if s["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(-1, keepdim=True))
        score = e / e.sum(-1, keepdim=True)
    key = score if s["bias"] is None else score + s["bias"]
    if s["groups"] > 1:
        by = key.view(key.shape[0], s["groups"], -1)
        best = by.sort(dim=-1, descending=True).values[..., :s["group_best"]].sum(-1)
        kept = best.sort(dim=-1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        key = torch.where(keep[..., None], by, float("-inf")).reshape(key.shape)
    experts = key.sort(dim=-1, descending=True, stable=True).indices[:, :s["k"]]
    weights = score.gather(1, experts)
    weights = weights / weights.sum(-1, keepdim=True) * s["scale"]
    return [weights, experts.to(torch.int32)]


def _plain_dispatch(s):
    rows, offsets, order = _rows_of(s["experts"], s["e"])
    routed = s["x"][order // s["experts"].shape[1]]
    live = torch.arange(routed.shape[0], device=routed.device) < offsets[-1]
    return [torch.where(live[:, None], routed, 0.0), offsets.to(torch.int32), rows.to(torch.int32)]


def _plain_combine(s):
    rows = s["rows"].long()
    y = torch.where((rows >= 0)[..., None], s["y"][rows.clamp(min=0)].float() * s["weights"][..., None], 0.0)
    out = y.sum(1)
    if s["base"] is not None:
        out = out + s["base"].float()
    return out.to(s["y"].dtype)


def _own(s):
    import w4a16_weight_only_gb300 as awq
    op = s["op"]
    if op == "rope":
        return list(awq.awq_rope(s["q"], s["k"], s["positions"], s["table"], interleaved=s["interleaved"]))
    if op == "rope_append":
        q = awq.awq_rope_append(s["q"], s["k"], s["v"], s["positions"], s["table"], s["k_cache"], s["v_cache"], s["slots"],
                                interleaved=s["interleaved"])
        return [q, s["k_cache"], s["v_cache"]]
    if op == "attention":
        return awq.awq_attention_shared(s["q"], s["k_cache"], s["v_cache"], s["prefix_pages"], s["prefix_len"], s["pages"],
                                        s["lens"], scale=s["scale"], max_len=s["max_len"])
    if op == "route":
        return list(awq.awq_moe_route(s["logits"], s["k"], scoring=s["scoring"], bias=s["bias"], groups=s["groups"],
                                      topk_groups=s["topk_groups"], group_best=s["group_best"], renormalize=True,
                                      scale=s["scale"]))
    if op == "dispatch":
        return list(awq.awq_moe_dispatch(s["x"], s["experts"], s["e"]))
    return awq.awq_moe_combine(s["y"], s["weights"], s["rows"], base=s["base"])


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "rope_append": _plain_rope, "attention": _plain_attention, "route": _plain_route,
            "dispatch": _plain_dispatch, "combine": _plain_combine}[state["op"]](state)


# ------------------------------------------------------------------------------------ work ----

def work(case):
    c, size = case, BYTES[case["dtype"]]
    if c["op"] in ("rope", "rope_append"):
        heads = c["hq"] + c["hkv"] * (2 if c["op"] == "rope_append" else 1)
        return {"bytes": c["t"] * (2 * heads * c["d"] * size + 4 * c["rot"] + 8),
                "flops": 3 * c["t"] * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] == "attention":
        lens, n, width = _lens(c), c["n"], c["hkv"] * c["d"]
        keys = c["prefix"] + sum(lens)
        pairs = c["b"] * n * c["prefix"] + sum(max(0, x - n + i + 1) for x in lens for i in range(n))
        return {"bytes": 2 * keys * width * size + 2 * c["b"] * n * c["hq"] * c["d"] * size + 4 * keys // c["page"],
                "flops": 4 * pairs * c["hq"] * c["d"]}
    if c["op"] == "route":
        return {"bytes": c["t"] * (c["e"] * size + 8 * c["k"]) + (4 * c["e"] if c["bias"] else 0), "flops": 8 * c["t"] * c["e"]}
    if c["op"] == "dispatch":
        return {"bytes": c["t"] * ((1 + c["k"]) * c["w"] * size + 8 * c["k"]) + 4 * (c["e"] + 1), "flops": 0}
    live = c["t"] * c["k"] * (1 - c["dropped"])
    return {"bytes": int((live + c["t"] * (2 if c["base"] else 1)) * c["w"] * size) + 8 * c["t"] * c["k"],
            "flops": int(2 * live * c["w"])}


# ----------------------------------------------------------------------------------- exact ----

def _exact_rope(c, s):
    f, factor = _frequencies(c["rot"], c["scaling"])
    turn = torch.polar(torch.full_like(f, factor)[None], s["positions"].double()[:, None] * f[None])[:, None]  # factor * e^(i angle)

    def rotated(x):
        x, rot = x.double().clone(), c["rot"]
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q, k = rotated(s["q"]), rotated(s["k"])
    if c["op"] == "rope":
        return [q, k]
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    for cache, x in zip(caches, (k, s["v"].double())):
        cells = cache.view(-1, c["hkv"], c["d"])
        for token, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                cells[slot] = x[token]
    return [q, *caches]


def _exact_attention(c, s):
    hkv, group, page, out = c["hkv"], c["hq"] // c["hkv"], c["page"], []
    gather = lambda cache, table, count: cache[table.long()].reshape(-1, hkv, c["d"])[:count].double()  # noqa: E731
    shared = [gather(s[x], s["prefix_pages"], c["prefix"]) for x in ("k_cache", "v_cache")]
    for i, count in enumerate(s["lens"].tolist()):
        k, v = (torch.cat([p, gather(s[x], s["pages"][i, :-(-count // page)], count)]) for p, x in zip(shared, ("k_cache", "v_cache")))
        q = s["q"][i].double().view(c["n"], hkv, group, c["d"])
        z = torch.einsum("nhgd,jhd->nhgj", q, k) / math.sqrt(c["d"])
        last = c["prefix"] + count - c["n"] + torch.arange(c["n"], device=z.device)
        z.masked_fill_(torch.arange(k.shape[0], device=z.device)[None, None, None] > last[:, None, None, None], float("-inf"))
        out.append(torch.einsum("nhgj,jhd->nhgd", torch.softmax(z, dim=-1), v).reshape(c["n"], c["hq"], c["d"]))
    return torch.stack(out)


def _exact_route(c, s):
    score, key, _ = _keys64(s["logits"], s["bias"], c)
    experts = key.sort(dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    weights = score.gather(1, experts)
    return [weights * (s["scale"] / weights.sum(-1, keepdim=True)), experts.to(torch.int32)]


def _exact_dispatch(c, s):
    ids = s["experts"].reshape(-1)
    offsets, routed, rows, done = [0], torch.zeros((ids.numel(), c["w"]), dtype=torch.float64, device="cuda"), torch.full_like(ids, -1), 0
    for e in range(c["e"]):
        places = (ids == e).nonzero()[:, 0]
        count = places.numel()
        routed[done:done + count] = s["x"][places // c["k"]].double()
        rows[places] = torch.arange(done, done + count, device="cuda", dtype=torch.int32)
        done += count
        offsets.append(done)
    return [routed, torch.tensor(offsets, dtype=torch.int32, device="cuda"), rows.view(s["experts"].shape)]


def _exact_combine(c, s):
    out = s["base"].double().clone() if s["base"] is not None else torch.zeros((c["t"], c["w"]), dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        live = s["rows"][:, j] >= 0
        out[live] += s["weights"][live, j].double()[:, None] * s["y"][s["rows"][live, j].long()].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "rope_append": _exact_rope, "attention": _exact_attention, "route": _exact_route,
            "dispatch": _exact_dispatch, "combine": _exact_combine}[case["op"]](case, s)
