"""awq_attention_shared where the prefix takes the tensor cores (more than 32 rows per key/value head): three
kernels, two of them side by side.  Graphs, streams, many row tiles, pages and offsets out of the ordinary.

Tolerances: the bound of test_gpu_attention.py."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


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


def make(B, n, hq, hkv, D, prefix, private, page, dtype=torch.float16, seed=0):
    """Ragged own lengths n .. private; NaN wherever no token was written."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = torch.randint(n, private + 1, (B,), generator=g, device="cuda")
    shared, per = -(-prefix // page), -(-private // page)
    order = torch.randperm(shared + B * per + 1, generator=g, device="cuda")
    pp, pages = order[:shared], order[shared:shared + B * per].view(B, per)
    live = torch.zeros((order.numel(), page), dtype=torch.bool, device="cuda")
    live[pp] = (torch.arange(shared * page, device="cuda") < prefix).view(shared, page)
    live[pages.reshape(-1)] = (torch.arange(per * page, device="cuda")[None] < lens[:, None]).view(B * per, page)
    k, v = (torch.randn((order.numel(), page, hkv, D), generator=g, device="cuda").to(dtype).masked_fill_(
        ~live[..., None, None], float("nan")) for _ in range(2))
    q = (1.5 * torch.randn((B, n, hq, D), generator=g, device="cuda")).to(dtype)
    return dict(q=q, k_cache=k, v_cache=v, prefix_pages=pp.int(), prefix_len=prefix, pages=pages.int(), lens=lens.int())


def check(out, d, sequences=None):
    q, k, v, prefix = d["q"], d["k_cache"], d["v_cache"], d["prefix_len"]
    B, n, hq, D = q.shape
    hkv, scale, u = k.shape[2], 1 / math.sqrt(D), U[q.dtype]
    pk, pv = (x[d["prefix_pages"].long()].reshape(-1, hkv, D)[:prefix].double() for x in (k, v))
    lens = d["lens"].tolist()
    for b in range(B) if sequences is None else sequences:
        kk, vv = (torch.cat([p, x[d["pages"][b].long()].reshape(-1, hkv, D)[:lens[b]].double()]) for p, x in ((pk, k), (pv, v)))
        qb = q[b].double().view(n, hkv, hq // hkv, D)
        z = scale * torch.einsum("nhgd,jhd->nhgj", qb, kk)
        size = float((scale * torch.einsum("nhgd,jhd->nhgj", qb.abs(), kk.abs())).max())
        last = prefix + lens[b] - n + torch.arange(n, device="cuda")
        z.masked_fill_(torch.arange(z.shape[-1], device="cuda") > last[:, None, None, None], float("-inf"))
        w = torch.softmax(z, dim=-1)
        want, spread = (torch.einsum("nhgj,jhd->nhgd", w, x).reshape(n, hq, D) for x in (vv, vv.abs()))
        fp32 = 2 * 2.0 ** -22 * (D + 8) * size + 2.0 ** -22 * (z.shape[-1] + 64)
        tol = u * want.abs() + (u + fp32) * spread * (1 + u) + 2.0 ** -24
        assert ((out[b].double() - want).abs() <= tol).all(), b


@pytest.mark.parametrize("rows", ["one tile more than 152, its second half empty", "160 tiles, several heads"])
def test_more_row_tiles_than_multiprocessors(awq, rows):
    # a block then goes through the steps of one tile after another, tiles of one and of two halves among them
    B, n, hq, hkv, prefix = (3000, 1, 13, 1, 300) if rows.startswith("one") else (1280, 2, 32, 2, 700)
    d = make(B, n, hq, hkv, 64, prefix, n + 2, 16, torch.bfloat16, seed=1)
    out = awq.awq_attention_shared(**d)
    check(out, d, [*range(0, B, 37), *range(B - 8, B)])
    assert torch.equal(awq.awq_attention_shared(**d), out)


def test_graph_with_new_values(awq):
    # lengths that move the split of the multiprocessors, too: none, few, all
    ds = [make(70, 1, 16, 2, 128, 1300, 400, 16, seed=s) for s in (2, 3, 4)]
    ds[1]["lens"].zero_()
    ds[2]["lens"].clamp_(max=3)
    want = [awq.awq_attention_shared(**d) for d in ds]
    for w, d in zip(want, ds):
        check(w, d, range(0, 70, 9))
    held = {n: t.clone() if torch.is_tensor(t) else t for n, t in ds[0].items()}
    out, s = torch.empty_like(held["q"]), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        awq.awq_attention_shared(**held, out=out)  # the stream's workspace exists
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(3):
                awq.awq_attention_shared(**held, out=out)
    torch.cuda.synchronize()
    for _ in range(4):
        for d, w in zip(ds, want):
            for name in ("q", "k_cache", "v_cache", "prefix_pages", "pages", "lens"):
                held[name].copy_(d[name])
            out.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, w)


def test_streams_and_graph_at_a_time(awq):
    ds = [make(70, 1, 16, 2, 128, 1300, 400, 16, seed=5), make(33, 2, 8, 1, 64, 3000, 900, 32, seed=6),
          make(100, 1, 8, 4, 96, 500, 60, 20, torch.bfloat16, seed=7)]
    want = [awq.awq_attention_shared(**d) for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    out, s = torch.empty_like(ds[0]["q"]), torch.cuda.Stream()
    workspace = torch.empty((awq.awq_attention_shared_workspace_size(70, 1, 16, 2, 128, 1300, ds[0]["pages"].shape[1] * 16),),
                            dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            awq.awq_attention_shared(**ds[0], out=out, workspace=workspace)
    got, replayed = [[] for _ in ds], []
    for _ in range(20):
        for stream, d, g in zip(streams, ds, got):
            with torch.cuda.stream(stream):
                g.append(awq.awq_attention_shared(**d))
        with torch.cuda.stream(s):
            graph.replay()
            replayed.append(out.clone())
    torch.cuda.synchronize()
    for w, g in zip([*want, want[0]], [*got, replayed]):
        assert all(torch.equal(x, w) for x in g)


def test_one_call_behind_another(awq):
    # the same workspace from call to call, sizes and splits in turn
    ds = [make(70, 1, 16, 2, 128, 1300, 400, 16, seed=8), make(40, 1, 8, 2, 128, 70, 3, 16, seed=9),
          make(3, 1, 8, 2, 128, 500, 700, 16, seed=10), make(64, 1, 8, 1, 64, 9000, 30, 64, seed=11)]
    want = [awq.awq_attention_shared(**d).clone() for d in ds]
    torch.cuda.synchronize()
    got = [awq.awq_attention_shared(**ds[i % 4]) for i in range(80)]
    assert all(torch.equal(g, want[i % 4]) for i, g in enumerate(got))
    for w, d in zip(want, ds):
        check(w, d, range(0, d["q"].shape[0], 9))


@pytest.mark.parametrize("page", [16, 20, 128])
def test_pages_outside_the_cache(awq, page):
    # by TMA boxes and by 16-byte copies: unspecified values, no access outside the cache
    d = make(50, 1, 8, 2, 64, 700, 300, page, seed=12)
    want = awq.awq_attention_shared(**d)
    own = dict(d, pages=d["pages"].clone())
    own["pages"][7, 0], own["pages"][9, -1] = -5, 1 << 30
    got = awq.awq_attention_shared(**own)
    rest = [b for b in range(50) if b not in (7, 9)]
    assert torch.equal(got[rest], want[rest])
    shared = dict(d, prefix_pages=d["prefix_pages"].clone())
    shared["prefix_pages"][0], shared["prefix_pages"][2], shared["prefix_pages"][-1] = 1 << 30, -1, d["k_cache"].shape[0]
    awq.awq_attention_shared(**shared)
    awq.device_status()
    assert torch.equal(awq.awq_attention_shared(**d), want)


@pytest.mark.parametrize("page", [16, 20])
def test_cache_offsets_past_32_bits(awq, page):
    d = make(40, 1, 4, 1, 128, 400, 60, page, seed=13)
    want = awq.awq_attention_shared(**d)
    used = d["k_cache"].shape[0]
    pages = (1 << 32) // (page * 128) + used
    for name in ("k_cache", "v_cache"):
        big = torch.empty((pages, page, 1, 128), dtype=torch.float16, device="cuda")
        big[-used:] = d[name]
        d[name] = big
    d["prefix_pages"] = d["prefix_pages"] + (pages - used)
    d["pages"] = d["pages"] + (pages - used)
    assert torch.equal(awq.awq_attention_shared(**d), want)


@pytest.mark.parametrize("rows", [32, 33, 128, 129, 256, 257])
def test_row_counts_around_the_tiles(awq, rows):
    # 32 rows stream, 33 take the tensor cores; halves and tiles that are just full
    for page in (16, 24):
        d = make(rows, 1, 2, 2, 128, 333, 40, page, seed=rows)
        check(awq.awq_attention_shared(**d), d, [*range(0, rows, 7), rows - 1])
