"""GPU parity of expert routing, dispatch and combine against the 64-bit oracle.

Experts, rows and offsets have to be equal; routing inputs leave out rows whose choice hangs on a
difference that 32-bit scores cannot hold.  Weights: exp and the divisions are good to a few ulp and a
sum over E terms to E 2^-24, so a relative 2^-23 (E + 16) bounds them.  Combine: one rounding of the
result (u |y|) and one fp32 rounding per product and sum, (2 k + 2) 2^-24 sum |terms|."""
import numpy as np
import pytest
import torch

from oracle import layer

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
U = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def awq():
    from w4a16_weight_only_gb300 import build
    build.build()
    import w4a16_weight_only_gb300 as awq
    assert awq.runtime_available(), awq.last_error()
    return awq


def f64(t):
    return t.detach().cpu().double().numpy()


def check_route(awq, logits, k, **kw):
    E = logits.shape[1]
    bias = kw.get("bias")
    want_w, want_e, clear = layer.moe_route(f64(logits), k, **{**kw, "bias": None if bias is None else f64(bias)})
    w, e = awq.awq_moe_route(logits, k, **kw)
    assert w.dtype is torch.float32 and e.dtype is torch.int32
    assert clear.mean() > 0.5
    assert np.array_equal(e.cpu().numpy()[clear], want_e[clear])
    err = np.abs(f64(w) - want_w)[clear]
    assert (err <= 2.0 ** -23 * (E + 16) * np.abs(want_w[clear])).all()
    return w, e


# E, k, groups, topk_groups, group_best: one expert, odd counts, groups of every kind of run, the most
ROUTES = [(1, 1, 1, 1, 1), (8, 2, 1, 1, 1), (60, 4, 1, 1, 1), (160, 6, 8, 3, 2), (256, 8, 8, 4, 2), (256, 32, 8, 8, 1),
          (33, 5, 3, 2, 2), (12, 3, 12, 3, 2), (96, 4, 32, 5, 1), (384, 8, 1, 1, 1), (512, 9, 4, 1, 2), (1024, 32, 16, 7, 2)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,topk_groups,group_best", ROUTES)
def test_route(awq, E, k, groups, topk_groups, group_best, scoring, dtype):
    g = torch.Generator().manual_seed(E + k)
    for T, biased in ((1, True), (37, False), (6, True)):
        logits = (1.5 * torch.randn((T, E), generator=g)).to(DT[dtype]).cuda()
        bias = (0.2 * torch.randn((E,), generator=g)).cuda() if biased else None
        if T == 1:  # leave a single row only if it is clear
            _, _, clear = layer.moe_route(f64(logits), k, scoring=scoring, bias=f64(bias), groups=groups,
                                          topk_groups=topk_groups, group_best=group_best)
            if not clear.all():
                continue
        check_route(awq, logits, k, scoring=scoring, bias=bias, groups=groups, topk_groups=topk_groups, group_best=group_best,
                    renormalize=T != 6, scale=2.5)


@pytest.mark.parametrize("E,groups", [(8, 1), (64, 1), (100, 1), (256, 8), (40, 5)])
def test_route_ties_go_to_the_lowest_index(awq, E, groups):
    rng = np.random.default_rng(E)
    logits = torch.from_numpy(rng.integers(-2, 3, (50, E)).astype(np.float32)).cuda()  # five values: ties everywhere
    logits[0] = 0.0
    logits[1] = torch.where(torch.arange(E) % 2 == 0, 0.0, -0.0).cuda()  # +0 and -0 are equal
    check_route(awq, logits, min(8, E // groups), groups=groups, topk_groups=max(1, groups // 2), group_best=1)


def test_route_experts_taken_out(awq):
    inf = float("inf")
    logits = torch.randn((6, 64), generator=torch.Generator().manual_seed(3)).cuda()
    logits[0] = -inf                       # nobody left
    logits[1, 3:] = -inf                   # fewer than k
    logits[2, :32] = -inf                  # whole groups
    logits[3, ::2] = -inf
    bias = torch.full((64,), 5.0, device="cuda")
    for scoring in ("softmax", "sigmoid"):
        for kw in (dict(), dict(groups=8, topk_groups=4, group_best=2)):
            w, e = check_route(awq, logits, 4, scoring=scoring, bias=bias, **kw)
            assert e[0].tolist() == [-1] * 4 and w[0].tolist() == [0] * 4 and e[1, 3] == -1 and w[1, 3] == 0


def test_route_extremes(awq):
    inf, nan = float("inf"), float("nan")
    logits = torch.zeros((5, 40), device="cuda")
    logits[0, 7] = nan
    logits[1, 9] = inf                     # softmax: inf - inf
    logits[2] = torch.finfo(torch.float32).min
    logits[3, :] = -200.0
    logits[4, 5] = 3e38
    w, e = awq.awq_moe_route(logits, 3)
    assert w[:2].isnan().all() and e[:2].tolist() == [[0, 1, 2]] * 2
    assert torch.allclose(w[2:4], torch.full((2, 3), 1 / 3, device="cuda"))
    assert e[4].tolist() == [5, 0, 1] and w[4].tolist() == [1, 0, 0]
    w, e = awq.awq_moe_route(logits, 3, scoring="sigmoid")
    assert w[0].isnan().all() and e[1].tolist() == [9, 0, 1] and torch.allclose(w[1], torch.tensor([0.5, 0.25, 0.25]).cuda())
    assert w[2].tolist() == [0, 0, 0] and e[2].tolist() == [0, 1, 2]  # scores of zero: no weight rather than 0 / 0


def test_route_strided_rows_and_out(awq):
    wide = torch.randn((9, 80), generator=torch.Generator().manual_seed(4)).half().cuda()
    for view in (wide[:, :64], wide[:, 3:67], wide[::2, 8:72]):
        w, e = check_route(awq, view, 6)
        out = (torch.empty_like(w), torch.empty_like(e))
        got = awq.awq_moe_route(view, 6, out=out)
        assert got[0] is out[0] and torch.equal(out[0], w) and torch.equal(out[1], e)


def ids(T, k, E, seed, dropped=0.0):
    rng = np.random.default_rng(seed)
    e = np.stack([rng.permutation(max(E, k))[:k] for _ in range(T)]).astype(np.int32) % E if T else np.zeros((0, k), np.int32)
    e[rng.random(e.shape) < dropped] = rng.choice([-1, E, 2 ** 30, -2 ** 31])
    return e


# T, k, E, W, dropped: one place, one expert, rows of odd width, all dropped, several blocks of the sort
DISPATCH = [(1, 1, 1, 8, 0.0), (13, 2, 8, 256, 0.0), (5, 3, 4, 33, 0.4), (64, 8, 60, 40, 0.1), (1000, 1, 3, 16, 0.0),
            (700, 6, 4096, 8, 0.3), (6, 2, 5, 64, 1.0), (5000, 8, 256, 8, 0.05), (2049, 2, 2, 7, 0.0), (3, 40, 64, 24, 0.2)]


@pytest.mark.parametrize("T,k,E,W,dropped", DISPATCH)
def test_dispatch(awq, T, k, E, W, dropped):
    e = ids(T, k, E, T + k, dropped)
    x = torch.randn((T, W + 3), generator=torch.Generator().manual_seed(T)).half().cuda()
    for view in (x[:, :W].contiguous(), x[:, :W], x[:, 3:]):
        routed, offsets, rows = awq.awq_moe_dispatch(view, torch.from_numpy(e).cuda(), E)
        want = layer.moe_dispatch(view.cpu().numpy(), e, E)
        assert np.array_equal(offsets.cpu().numpy(), want[1]) and np.array_equal(rows.cpu().numpy(), want[2])
        assert np.array_equal(routed.cpu().numpy().view(np.uint16), want[0].view(np.uint16))


def test_dispatch_many_places(awq):
    # more places than 128 blocks of 1024: the blocks' parts grow
    T, k, E = 70001, 4, 64
    e = ids(997, k, E, 1, 0.1)[np.random.default_rng(2).integers(0, 997, T)]
    x = torch.arange(T, device="cuda", dtype=torch.int32).view(torch.float16).view(T, 2)
    routed, offsets, rows = awq.awq_moe_dispatch(x, torch.from_numpy(e).cuda(), E)
    flat = np.where((e >= 0) & (e < E), e, E).reshape(-1)
    order = np.argsort(flat, kind="stable")
    live = int((flat < E).sum())
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E + 1)[:E])]))
    place = np.empty_like(order)
    place[order] = np.arange(order.size)
    assert np.array_equal(rows.cpu().numpy().reshape(-1), np.where(flat < E, place, -1))
    got = routed.view(torch.int32).cpu().numpy()[:, 0]
    assert np.array_equal(got[:live], (order // k)[:live]) and not got[live:].any()


def test_dispatch_empty(awq):
    x, e = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda")
    routed, offsets, rows = awq.awq_moe_dispatch(x, e, 5)
    assert routed.shape == (0, 16) and offsets.tolist() == [0] * 6 and rows.shape == (0, 2)
    x, e = torch.empty((3, 0), dtype=torch.bfloat16, device="cuda"), torch.tensor([[1], [0], [1]], dtype=torch.int32, device="cuda")
    routed, offsets, rows = awq.awq_moe_dispatch(x, e, 2)
    assert routed.shape == (3, 0) and offsets.tolist() == [0, 1, 3] and rows.flatten().tolist() == [1, 0, 2]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,k,W,R,base", [(1, 1, 8, 1, False), (13, 2, 4096, 26, True), (5, 3, 33, 15, True), (64, 8, 520, 512, False),
                                          (3, 0, 16, 0, True), (4, 2, 24, 0, False), (200, 6, 72, 900, True), (2, 40, 2050, 80, False)])
def test_combine(awq, T, k, W, R, base, dtype):
    g = torch.Generator().manual_seed(T + W)
    y = torch.randn((R, W), generator=g).to(DT[dtype]).cuda()
    w = torch.rand((T, k), generator=g).cuda()
    rows = np.random.default_rng(W).integers(-1, R + 1, (T, k)).astype(np.int32)  # -1 and R: left out
    b = torch.randn((T, W), generator=g).to(DT[dtype]).cuda() if base else None
    out = awq.awq_moe_combine(y, w, torch.from_numpy(rows).cuda(), base=b)
    want, size = layer.moe_combine(f64(y), f64(w), rows, None if b is None else f64(b))
    tol = U[dtype] * np.abs(want) + (2 * k + 2) * 2.0 ** -24 * size + (2.0 ** -25 if dtype == "fp16" else 0)
    assert (np.abs(f64(out) - want) <= tol * (1 + 1e-6)).all()
    if base:
        assert torch.equal(awq.awq_moe_combine(y, w, torch.from_numpy(rows).cuda(), base=b, out=b), out)


def test_combine_leaves_out_rows_that_hold_nan(awq):
    y = torch.ones((3, 16), dtype=torch.float16, device="cuda")
    y[1] = float("nan")
    w = torch.tensor([[0.5, float("nan")]], device="cuda")
    out = awq.awq_moe_combine(y, w, torch.tensor([[2, -1]], dtype=torch.int32, device="cuda"))
    assert torch.equal(out, torch.full((1, 16), 0.5, dtype=torch.float16, device="cuda"))


def test_dispatch_combine_is_the_identity(awq):
    T, k, E, W = 300, 4, 32, 128
    x = torch.randn((T, W), generator=torch.Generator().manual_seed(1)).half().cuda()
    e = torch.from_numpy(ids(T, k, E, 5)).cuda()
    routed, _, rows = awq.awq_moe_dispatch(x, e, E)
    assert torch.equal(awq.awq_moe_combine(routed, torch.full((T, k), 0.25, device="cuda"), rows), x)


def test_on_other_streams(awq):
    # the same calls on two streams at a time, and the stream given by handle
    T, k, E, W = 3000, 4, 32, 256
    x = torch.randn((T, W), generator=torch.Generator().manual_seed(1)).half().cuda()
    es = [torch.from_numpy(ids(T, k, E, s)).cuda() for s in (1, 2)]
    want = [awq.awq_moe_dispatch(x, e, E) for e in es]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s, e in zip(streams, es):
            with torch.cuda.stream(s):
                got.append(awq.awq_moe_dispatch(x, e, E))
    outs = [tuple(torch.empty_like(t) for t in w) for w in want]
    torch.cuda.synchronize()
    awq.awq_moe_dispatch(x, es[0], E, out=outs[0], stream=streams[0])
    awq.awq_moe_dispatch(x, es[1], E, out=outs[1], stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    for i, g in enumerate(got + outs):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


def test_refusals(awq):
    x, e = torch.zeros((4, 16), dtype=torch.float16, device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        awq.awq_moe_dispatch(x, e.long(), 4)
    with pytest.raises(ValueError):
        awq.awq_moe_dispatch(x[:3], e, 4)
    with pytest.raises(ValueError):
        awq.awq_moe_dispatch(x.cpu(), e, 4)
    with pytest.raises(awq.AwqError):
        awq.awq_moe_dispatch(x, e, 4, workspace=torch.empty((16,), dtype=torch.uint8, device="cuda"))
    with pytest.raises(awq.AwqError):
        awq.awq_moe_dispatch(x, e, 5000)
    logits = torch.zeros((4, 16), device="cuda")
    with pytest.raises(TypeError):
        awq.awq_moe_route(logits.double(), 2)
    with pytest.raises(ValueError):
        awq.awq_moe_route(logits, 2, scoring="other")
    with pytest.raises(ValueError):
        awq.awq_moe_route(logits.t(), 2)
    with pytest.raises(TypeError):
        awq.awq_moe_route(logits, 2, bias=torch.zeros((16,), dtype=torch.float16, device="cuda"))
    with pytest.raises(awq.AwqError):
        awq.awq_moe_route(logits, 17)
    with pytest.raises(awq.AwqError):
        awq.awq_moe_route(logits, 2, groups=3)
    with pytest.raises(TypeError):
        awq.awq_moe_combine(x, torch.zeros((4, 2), dtype=torch.float16, device="cuda"), e)
    with pytest.raises(ValueError):
        awq.awq_moe_combine(x, torch.zeros((4, 3), device="cuda"), e)
    with pytest.raises(ValueError):
        awq.awq_moe_combine(x[:, ::2], torch.zeros((4, 2), device="cuda"), e)


@pytest.mark.parametrize("W", [65535 * 128 + 1, 65535 * 1024 + 8])
def test_rows_wider_than_a_grid_of_runs(awq, W):
    # one element or one vector of eight more than 65535 blocks of 128 threads take
    g = torch.Generator(device="cuda").manual_seed(W)
    x = torch.randint(-100, 100, (2, W), generator=g, device="cuda", dtype=torch.int32).half()
    routed, offsets, rows = awq.awq_moe_dispatch(x, torch.tensor([[1, 0], [0, -1]], dtype=torch.int32, device="cuda"), 2)
    assert offsets.tolist() == [0, 2, 3] and rows.tolist() == [[2, 0], [1, -1]]
    assert torch.equal(routed[:3], x[[0, 1, 0]]) and not routed[3].any()
    weights = torch.tensor([[0.5, 0.25], [2.0, 7.0]], device="cuda")
    out = awq.awq_moe_combine(routed, weights, rows, base=x)
    assert torch.equal(out, x * torch.tensor([[1.75], [3.0]], dtype=torch.float16, device="cuda"))


def test_sigmoid_weights_keep_their_last_bit(awq):
    # 1 / (1 + e), e = exp(-x): exp to one ulp (2^-23, moving the result by e / (1 + e) of that), a rounded sum
    # and a rounded quotient (2^-24 each)
    x = torch.linspace(-12.0, 25.0, 1 << 20, device="cuda").view(-1, 8)
    w, e = awq.awq_moe_route(x, 8, scoring="sigmoid", renormalize=False)
    got = torch.empty_like(w).scatter_(1, e.long(), w)
    big = torch.exp(-x.double())
    want = 1 / (1 + big)
    tol = (2.0 ** -23 * big / (1 + big) + 2.0 ** -23) * (1 + 2.0 ** -20)
    assert (((got.double() - want) / want).abs() <= tol).all()
