"""GPU parity of awq_attention_shared against the 64-bit oracle.

Tolerance, per element: the result's rounding u |y| (u = 2^-11 fp16, 2^-8 bf16); the probabilities'
rounding to the same type, at most u sum_j p_j |v_j|; and fp32 arithmetic: a logit is a sum of D
products (error at most 2^-22 (D + 8) Z, Z the largest scale * sum |q k|, which moves p by that
relative amount, twice through the denominator), and sums over N keys (2^-22 (N + 64) relative).  All
but the first are relative to sum_j p_j |v_j|."""
import math

import numpy as np
import pytest
import torch

from oracle import layer

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
U = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def awq():
    from w4a16_weight_only_gb300 import build
    build.build()
    import w4a16_weight_only_gb300 as awq
    assert awq.runtime_available(), awq.last_error()
    return awq


@pytest.fixture(autouse=True)
def no_wait_gave_up(awq):
    yield
    awq.device_status()


def f64(t):
    return t.detach().cpu().double().numpy()


def make(B, n, hq, hkv, D, prefix, lens, page, dtype, seed=0, sharp=1.0, layout="token", spare=0):
    """Inputs whose cache holds NaN wherever no token was written."""
    rng = np.random.default_rng(seed)
    per = max(1, -(-max(list(lens) + [1]) // page)) + spare
    shared = -(-prefix // page)
    total = shared + B * per + 2
    order = rng.permutation(total)
    pp, pages = order[:shared].astype(np.int32), order[shared:shared + B * per].reshape(B, per).astype(np.int32)
    k, v = (np.full((total, page, hkv, D), np.nan) for _ in range(2))
    for x in (k, v):
        for j in range(prefix):
            x[pp[j // page], j % page] = rng.standard_normal((hkv, D))
        for b in range(B):
            for j in range(lens[b]):
                x[pages[b, j // page], j % page] = rng.standard_normal((hkv, D))
    def cache(x):
        t = torch.from_numpy(x).to(DT[dtype])
        return t.cuda() if layout == "token" else t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    q = torch.from_numpy(sharp * rng.standard_normal((B, n, hq, D))).to(DT[dtype]).cuda()
    return dict(q=q, k_cache=cache(k), v_cache=cache(v), prefix_pages=torch.from_numpy(pp).cuda(), prefix_len=prefix,
                pages=torch.from_numpy(pages).cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def check(out, d, dtype, scale=None):
    D = d["q"].shape[-1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    q = f64(d["q"]) if d["q"].dim() == 4 else f64(d["q"])[:, None]
    lens = d["lens"].tolist()
    want, spread, z = layer.attention_shared(q, f64(d["k_cache"]), f64(d["v_cache"]), d["prefix_pages"].tolist(),
                                             d["prefix_len"], d["pages"].tolist(), lens, scale)
    N = d["prefix_len"] + max(lens + [0])
    fp32 = 2 * 2.0 ** -22 * (D + 8) * z + 2.0 ** -22 * (N + 64)
    tol = U[dtype] * np.abs(want) + (U[dtype] + fp32) * spread * (1 + U[dtype]) + (2.0 ** -24 if dtype == "fp16" else 0)
    err = np.abs(f64(out).reshape(want.shape) - want)
    assert np.isfinite(f64(out)).all()
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())


# B, n, hq, hkv, D, prefix, lens, page
CASES = [
    (1, 1, 1, 1, 64, 1, [1], 16),                       # one key each
    (1, 1, 8, 8, 128, 0, [1], 16),                      # no prefix
    (2, 1, 8, 2, 128, 37, [0, 0], 16),                  # no private keys
    (3, 1, 8, 1, 128, 129, [5, 0, 200], 16),            # a sequence without keys of its own among others
    (2, 1, 4, 4, 128, 300, [17, 64], 20),               # pages that end inside a tile
    (4, 1, 16, 2, 64, 511, [1, 15, 16, 33], 7),
    (2, 3, 6, 2, 96, 100, [3, 50], 16),                 # several new tokens, causal
    (2, 5, 14, 2, 128, 65, [5, 131], 1),                # pages of one token
    (1, 1, 64, 1, 128, 260, [90], 64),                  # one key/value head for all
    (2, 2, 40, 1, 64, 33, [2, 34], 32),                 # more than 64 rows a sequence
    (2, 1, 8, 2, 256, 150, [31, 70], 16),
    (1, 20, 4, 4, 256, 19, [40], 16),
    (33, 1, 8, 2, 128, 257, [(7 * i) % 41 for i in range(33)], 16),   # 132 rows over the prefix
    (70, 1, 4, 1, 64, 640, [(5 * i) % 23 for i in range(70)], 16),    # 280 rows
    (12, 3, 16, 2, 128, 1025, [3 + (11 * i) % 90 for i in range(12)], 128),  # 288 rows
    (1, 1, 2, 1, 128, 6000, [10], 16),                  # a long prefix, few rows: cut along the keys
    (1, 1, 2, 1, 128, 16, [5000], 16),                  # a long private part
    (40, 4, 4, 1, 96, 130, [4 + i % 9 for i in range(40)], 16),       # many rows, the other head sizes
    (20, 4, 4, 1, 256, 130, [4 + i % 9 for i in range(20)], 16),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(awq, case, dtype):
    B, n, hq, hkv, D, prefix, lens, page = CASES[case]
    d = make(B, n, hq, hkv, D, prefix, lens, page, dtype, seed=case)
    check(awq.awq_attention_shared(**d), d, dtype)
    assert torch.equal(awq.awq_attention_shared(**d), awq.awq_attention_shared(**d))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B,n,hq,hkv,D,prefix,private,page", [
    (300, 1, 32, 16, 64, 2565, 40, 16),    # several steps of several tiles per block, the prefix's end among them
    (75, 2, 32, 8, 128, 4097, 100, 32),
    (130, 1, 16, 16, 96, 3000, 33, 24),    # pages that no TMA box divides
    (64, 1, 64, 8, 128, 5000, 50, 128),
    (48, 1, 8, 2, 128, 300, 3000, 16),     # own keys outweigh the prefix: most SMs stream
])
def test_many_rows(awq, B, n, hq, hkv, D, prefix, private, page, dtype):
    g = torch.Generator(device="cuda").manual_seed(B)
    lens = torch.randint(n, private + 1, (B,), generator=g, device="cuda")
    shared, per = -(-prefix // page), -(-private // page)
    order = torch.randperm(shared + B * per + 1, generator=g, device="cuda")
    pp, pages = order[:shared], order[shared:shared + B * per].view(B, per)
    live = torch.zeros((order.numel(), page), dtype=torch.bool, device="cuda")
    live[pp] = (torch.arange(shared * page, device="cuda") < prefix).view(shared, page)
    live[pages.reshape(-1)] = (torch.arange(per * page, device="cuda")[None] < lens[:, None]).view(B * per, page)
    k, v = (torch.randn((order.numel(), page, hkv, D), generator=g, device="cuda").to(DT[dtype]).masked_fill_(
        ~live[..., None, None], float("nan")) for _ in range(2))
    q = (1.5 * torch.randn((B, n, hq, D), generator=g, device="cuda")).to(DT[dtype])
    out = awq.awq_attention_shared(q, k, v, pp.int(), prefix, pages.int(), lens.int()).double()
    scale, group, zmax = 1 / math.sqrt(D), hq // hkv, 0.0
    pk, pv = (x[pp].reshape(-1, hkv, D)[:prefix].double() for x in (k, v))
    for b in range(B):
        count = int(lens[b])
        kk, vv = (torch.cat([p, x[pages[b]].reshape(-1, hkv, D)[:count].double()]) for p, x in ((pk, k), (pv, v)))
        qb = q[b].double().view(n, hkv, group, D)
        z = scale * torch.einsum("nhgd,jhd->nhgj", qb, kk)
        if b == 0:
            zmax = 1.5 * float((scale * torch.einsum("nhgd,jhd->nhgj", qb.abs(), kk.abs())).max())
        last = prefix + count - n + torch.arange(n, device="cuda")
        z.masked_fill_(torch.arange(z.shape[-1], device="cuda") > last[:, None, None, None], float("-inf"))
        w = torch.softmax(z, dim=-1)
        want, spread = (torch.einsum("nhgj,jhd->nhgd", w, x).reshape(n, hq, D) for x in (vv, vv.abs()))
        fp32 = 2 * 2.0 ** -22 * (D + 8) * zmax + 2.0 ** -22 * (prefix + private + 64)
        tol = U[dtype] * want.abs() + (U[dtype] + fp32) * spread * (1 + U[dtype]) + (2.0 ** -24 if dtype == "fp16" else 0)
        assert ((out[b] - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_sharp_distributions(awq, dtype):
    # logits of +-60: one key takes nearly all, and the running maximum moves far
    d = make(3, 1, 8, 2, 128, 700, [100, 3, 50], 16, dtype, seed=5, sharp=20.0)
    check(awq.awq_attention_shared(**d), d, dtype)
    d = make(40, 1, 8, 2, 128, 700, [10] * 40, 16, dtype, seed=6, sharp=20.0)
    check(awq.awq_attention_shared(**d), d, dtype)


def test_rows_that_see_nothing(awq):
    # without a prefix, new tokens beyond what the sequence holds, and an empty sequence
    d = make(3, 3, 4, 2, 64, 0, [1, 0, 5], 16, "fp16", seed=2)
    out = awq.awq_attention_shared(**d)
    check(out, d, "fp16")
    assert not out[0, :2].any() and not out[1].any() and out[0, 2].any()


def test_head_order_layout_strides_scale(awq):
    d = make(3, 2, 8, 4, 128, 90, [20, 2, 47], 20, "bf16", seed=3, layout="head")
    check(awq.awq_attention_shared(**d, scale=0.05), d, "bf16", 0.05)
    rows = torch.randn((3 * 2, 20 * 128), device="cuda").bfloat16()  # queries inside fused rows
    d["q"] = rows[:, :8 * 128].view(3, 2, 8, 128)
    check(awq.awq_attention_shared(**d), d, "bf16")
    d["q"] = rows.view(3, 2, 20, 128)[:, 1, 4:12]  # three dimensions: one token per sequence
    out = awq.awq_attention_shared(**d)
    assert out.shape == (3, 8, 128)
    check(out, d, "bf16")


def test_keys_and_values_side_by_side(awq):
    d = make(2, 1, 4, 2, 64, 50, [20, 9], 16, "fp16", seed=4)
    both = torch.stack([d["k_cache"], d["v_cache"]], dim=1)
    want = awq.awq_attention_shared(**d)
    d["k_cache"], d["v_cache"] = both[:, 0], both[:, 1]
    assert torch.equal(awq.awq_attention_shared(**d), want)


def test_max_len_bounds(awq):
    # a tighter bound gives the same values; a length above it is cut to it
    d = make(2, 1, 4, 2, 64, 50, [20, 9], 16, "fp16", seed=4, spare=40)
    check(awq.awq_attention_shared(**d, max_len=20), d, "fp16")
    check(awq.awq_attention_shared(**d, max_len=21), d, "fp16")
    cut = awq.awq_attention_shared(**d, max_len=12)
    d["lens"] = torch.tensor([12, 9], dtype=torch.int32, device="cuda")
    check(cut, d, "fp16")


def test_pages_outside_the_cache(awq):
    # unspecified values for that sequence only, and no access outside the cache
    d = make(3, 1, 4, 2, 64, 40, [33, 20, 7], 16, "fp16", seed=7)
    want = awq.awq_attention_shared(**d)
    d["pages"] = d["pages"].clone()
    d["pages"][1, 0] = -5
    d["pages"][1, 1] = 1 << 30
    got = awq.awq_attention_shared(**d)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


def test_values_of_infinity_and_nan_reach_only_their_rows(awq):
    d = make(2, 1, 4, 2, 64, 40, [33, 20], 16, "fp16", seed=8)
    want = awq.awq_attention_shared(**d)
    d["q"] = d["q"].clone()
    d["q"][0, 0, 1, 5] = float("nan")
    got = awq.awq_attention_shared(**d)
    assert got[0, 0, 1].isnan().all()
    got[0, 0, 1] = want[0, 0, 1]
    assert torch.equal(got, want)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("B,n,hq,hkv,D,prefix,lens,page", [
    (3, 4, 8, 1, 128, 0, [4, 21, 70], 16),
    (2, 2, 2, 1, 64, 100, [2, 16], 7),          # 4 rows a sequence, the prefix streamed
    (2, 3, 40, 2, 96, 150, [17, 3], 16),        # 60 rows a sequence, the prefix on the tensor cores
    (1, 20, 4, 4, 256, 19, [40], 16),
])
def test_values_of_newer_tokens_reach_only_rows_that_see_them(awq, B, n, hq, hkv, D, prefix, lens, page, value):
    for dtype in ("fp16", "bf16"):
        d = make(B, n, hq, hkv, D, prefix, lens, page, dtype, seed=13)
        finite = awq.awq_attention_shared(**d)
        e = dict(d, v_cache=d["v_cache"].clone())
        for b in range(B):  # the two newest tokens' values
            for j in (lens[b] - 1, lens[b] - 2):
                e["v_cache"][int(d["pages"][b, j // page]), j % page] = value
        got = awq.awq_attention_shared(**e)
        assert not got[:, n - 2:].isfinite().any()
        got[:, n - 2:] = finite[:, n - 2:]
        check(got, d, dtype)


def test_scale_of_zero_and_below(awq):
    for scale in (0.0, -0.05):
        for B in (3, 40):  # the prefix streamed, and on the tensor cores
            d = make(B, 1, 8, 2, 128, 300, [10] * B, 16, "fp16", seed=14)
            check(awq.awq_attention_shared(**d, scale=scale), d, "fp16", scale)


def test_keys_of_small_weight(awq):
    # every 16th key has the largest logit and a value of zero; the others, e^-13 of its weight (below
    # fp16's full precision), make the result
    for B in (2, 40):
        d = make(B, 1, 4, 1, 64, 608, [96] * B, 16, "fp16", seed=15)
        d["q"].zero_()
        d["q"][..., 0] = 1.0
        d["k_cache"][..., 0] = -13.0
        d["v_cache"].abs_().mul_(1000.0)
        d["k_cache"][:, 0, :, 0] = 0.0
        d["v_cache"][:, 0] = 0.0
        check(awq.awq_attention_shared(**d, scale=1.0), d, "fp16", 1.0)


def test_cache_offsets_past_32_bits(awq):
    d = make(2, 1, 4, 1, 256, 40, [33, 20], 16, "fp16", seed=9)
    want = awq.awq_attention_shared(**d)
    used = d["k_cache"].shape[0]
    pages = (1 << 32) // (16 * 256) + used
    for name in ("k_cache", "v_cache"):
        big = torch.empty((pages, 16, 1, 256), dtype=torch.float16, device="cuda")
        big[-used:] = d[name]
        d[name] = big
    d["prefix_pages"] = d["prefix_pages"] + (pages - used)
    d["pages"] = d["pages"] + (pages - used)
    assert torch.equal(awq.awq_attention_shared(**d), want)


def test_stacked_query_rows_past_32_bits(awq):
    # a batch stride that takes the second sequence's queries past 2^31 elements
    d = make(2, 1, 2, 1, 64, 20, [3, 4], 16, "bf16", seed=10)
    far = torch.empty(((1 << 31) + 1024,), dtype=torch.bfloat16, device="cuda")
    q = far.as_strided((2, 1, 2, 64), ((1 << 31) + 64, 128, 64, 1))
    q.copy_(d["q"])
    want = awq.awq_attention_shared(**d)
    d["q"] = q
    assert torch.equal(awq.awq_attention_shared(**d), want)


def test_graph_and_streams(awq):
    ds = [make(4, 1, 8, 2, 128, 300, [40, 3, 0, 77], 16, "fp16", seed=s) for s in (11, 12)]
    want = [awq.awq_attention_shared(**d) for d in ds]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s, d in zip(streams, ds):
            with torch.cuda.stream(s):
                got.append(awq.awq_attention_shared(**d))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 2]) for i, g in enumerate(got))
    out = torch.empty_like(ds[0]["q"])
    with torch.cuda.stream(streams[0]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            awq.awq_attention_shared(**ds[0], out=out)
    for d, w in zip(ds, want):  # new values in the captured tensors
        for name in ("q", "k_cache", "v_cache", "prefix_pages", "pages", "lens"):
            ds[0][name].copy_(d[name].clone())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


def test_refusals(awq):
    d = make(2, 1, 4, 2, 64, 40, [33, 20], 16, "fp16")
    bad = lambda **kw: awq.awq_attention_shared(**{**d, **kw})  # noqa: E731
    with pytest.raises(TypeError):
        bad(q=d["q"].float())
    with pytest.raises(TypeError):
        bad(q=d["q"].bfloat16())
    with pytest.raises(ValueError):
        bad(prefix_len=49)
    with pytest.raises(ValueError):
        bad(lens=d["lens"][:1])
    with pytest.raises(TypeError):
        bad(lens=d["lens"].long())
    with pytest.raises(ValueError):
        bad(pages=d["pages"].cpu())
    with pytest.raises(ValueError):
        bad(q=torch.zeros((4, 64), dtype=torch.float16, device="cuda"))
    with pytest.raises(awq.AwqError):
        bad(q=torch.zeros((2, 1, 3, 64), dtype=torch.float16, device="cuda"))
    with pytest.raises(awq.AwqError):
        bad(max_len=10 ** 6)
    with pytest.raises(awq.AwqError):
        bad(workspace=torch.empty((256,), dtype=torch.uint8, device="cuda"))
    with pytest.raises(awq.AwqError):
        bad(q=torch.zeros((2, 1, 4, 80), dtype=torch.float16, device="cuda"),
            k_cache=torch.zeros((9, 16, 2, 80), dtype=torch.float16, device="cuda"),
            v_cache=torch.zeros((9, 16, 2, 80), dtype=torch.float16, device="cuda"))


def test_empty(awq):
    d = make(2, 1, 4, 2, 64, 40, [33, 20], 16, "fp16")
    d.update(q=d["q"][:0], pages=d["pages"][:0], lens=d["lens"][:0])
    assert awq.awq_attention_shared(**d).shape == (0, 1, 4, 64)


# B, n, hq, hkv, D, prefix, lens, page, workspace's content; every call has streaming warps that wait, the last
# two blocks of the prefix kernel with several steps as well
GIVE_UPS = [
    (2, 1, 8, 2, 128, 300, [40, 33], 16),
    (3, 1, 4, 2, 64, 0, [200, 1, 90], 16),
    (2, 20, 4, 4, 256, 64, [40, 64], 32),
    (40, 1, 8, 1, 128, 128 * 900, [20] * 40, 64),
    (70, 2, 8, 1, 64, 128 * 640 + 5, [50] * 70, 128),
]


@pytest.mark.parametrize("word", [0x4f3a1200, 0x7fffffff, -1, -(1 << 31)])
@pytest.mark.parametrize("case", range(len(GIVE_UPS)))
def test_waits_that_give_up_are_reported(awq, case, word):
    # nothing arrives in time: an error status, whatever the workspace held, and the next call is right
    B, n, hq, hkv, D, prefix, lens, page = GIVE_UPS[case]
    g = torch.Generator(device="cuda").manual_seed(case)
    shared, per = -(-prefix // page), -(-max(lens) // page)
    order = torch.randperm(shared + B * per, generator=g, device="cuda", dtype=torch.int32)
    k, v = (torch.randn((order.numel(), page, hkv, D), generator=g, device="cuda").half() for _ in range(2))
    d = dict(q=torch.randn((B, n, hq, D), generator=g, device="cuda").half(), k_cache=k, v_cache=v, prefix_pages=order[:shared],
             prefix_len=prefix, pages=order[shared:].view(B, per), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    want = awq.awq_attention_shared(**d)
    size = awq.awq_attention_shared_workspace_size(B, n, hq, hkv, D, prefix, per * page)
    workspace = torch.full((-(-size // 4),), word, dtype=torch.int32, device="cuda").view(torch.uint8)
    awq.device_status()
    awq.selftest_attention_give_up(True)
    try:
        awq.awq_attention_shared(**d, workspace=workspace)
    finally:
        awq.selftest_attention_give_up(False)
    with pytest.raises(awq.AwqError, match="bounded wait"):
        awq.device_status()
    assert torch.equal(awq.awq_attention_shared(**d, workspace=workspace), want)


def test_strides_of_single_entries_do_not_matter(awq):
    # one sequence of one token inside rows of odd length; one head whose stride differs between keys and values
    d = make(1, 1, 2, 1, 64, 50, [20], 16, "fp16", seed=21)
    want = awq.awq_attention_shared(**d)
    e = dict(d, q=d["q"].as_strided((1, 1, 2, 64), (131, 257, 64, 1)))
    pages = d["k_cache"].shape[0]
    e["v_cache"] = d["v_cache"].as_strided((pages, 16, 1, 64), (1024, 64, 1024, 1))
    e["k_cache"] = d["k_cache"].as_strided((pages, 16, 1, 64), (1024, 64, 3, 1))
    assert torch.equal(awq.awq_attention_shared(**e), want)
    many = make(40, 1, 2, 1, 64, 300, [20] * 40, 16, "fp16", seed=22)  # the prefix on the tensor cores
    want = awq.awq_attention_shared(**many)
    pages = many["k_cache"].shape[0]
    many["k_cache"] = many["k_cache"].as_strided((pages, 16, 1, 64), (1024, 64, 3, 1))
    assert torch.equal(awq.awq_attention_shared(**many), want)
    table, cache = awq.awq_rope_table(16, 64), torch.zeros((2, 2, 16, 1, 64), dtype=torch.float16, device="cuda")
    k, slots = torch.randn((3, 1, 64), device="cuda").half(), torch.arange(3, dtype=torch.int32, device="cuda")
    awq.awq_rope_append(k, k, k, slots, table, cache[0].as_strided((2, 16, 1, 64), (1024, 64, 5, 1)), cache[1], slots)
    assert torch.equal(cache[1, 0, :3], k) and cache[0, 0, :3].any()


@pytest.mark.parametrize("B,n,hq,hkv,D,prefix,lens,page", [
    (3, 2, 4, 2, 64, 20, [2, 7, 40], 16),       # streamed
    (2, 1, 8, 2, 128, 0, [9, 30], 7),
    (40, 1, 4, 1, 128, 300, [10] * 40, 16),     # the prefix on the tensor cores
    (2, 20, 4, 4, 256, 19, [40, 20], 16),
])
def test_rows_whose_logits_are_all_minus_infinity(awq, B, n, hq, hkv, D, prefix, lens, page):
    # 0 / 0 by the definition, not the zero of a row that sees no key; one finite logit is enough
    for dtype in ("fp16", "bf16"):
        d = make(B, n, hq, hkv, D, prefix, lens, page, dtype, seed=17)
        d["q"][..., 0] = 1.0
        d["q"][0, 0, 0, 0] = 0.5
        d["k_cache"][..., 0] = float("-inf")
        out = awq.awq_attention_shared(**d)
        assert out.isnan().all()
        j = lens[0] - n  # a key that all rows of the first sequence see
        d["k_cache"][int(d["pages"][0, j // page]), j % page] = 0.25
        out = awq.awq_attention_shared(**d)
        assert out[1:].isnan().all()
        value = d["v_cache"][int(d["pages"][0, j // page]), j % page]
        assert torch.equal(out[0], value.repeat_interleave(hq // hkv, 0)[None].expand(n, hq, D))
