"""GPU parity of awq_residual_norm against the 64-bit oracle.

Tolerance, per element: the output's rounding u |y| (u = 2^-11 fp16, 2^-8 bf16; fp16 results below the normal
range round to a multiple of 2^-24), and the oracle's bound on fp32 arithmetic: sums of W numbers over at
least 256 threads (relative error at most 2^-22 (64 + W / 256)), carried through the root, the products and
the second norm to first order (doubled for the higher ones)."""
import numpy as np
import pytest
import torch

from oracle import step

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


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def inputs(T, W, dtype, seed, residual=True, post=False, gate="none", kind="rms", bias=False, weight=True, pad=0, mean=0.5):
    g = torch.Generator().manual_seed(seed)
    draw = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    to = lambda x: x.to(DT[dtype]).cuda()  # noqa: E731
    d = {"x": to(3.0 * draw(T, W + pad) + mean)[:, :W], "kind": kind}
    if residual:
        d["residual"] = to(10.0 * draw(T, W + 2 * pad))[:, :W]
    if weight:
        d["weight"] = to(1 + 0.1 * draw(W))
    if post:
        d["post_weight"] = to(1 + 0.1 * draw(W))
    if bias and weight:
        d["bias"] = to(0.1 * draw(W))
    if bias and post:
        d["post_bias"] = to(0.1 * draw(W))
    if gate != "none":
        d["gate"] = to(draw(W) if gate == "channel" else draw(T, W + pad)[:, :W])
    return d


def check(got, d, dtype, **kw):
    arrays = {k: f64(v) if torch.is_tensor(v) else v for k, v in d.items()}
    h, y, dh, dy = step.residual_norm(**arrays, **kw)
    for name, out, want, bound in (("h", got[0], h, dh), ("y", got[1], y, dy)):
        if want is None:
            assert out is None
            continue
        tol = U[dtype] * np.abs(want) + 2 * bound + (2.0 ** -24 if dtype == "fp16" else 0)
        err = np.abs(f64(out) - want)
        assert (err <= tol).all(), (name, float((err / tol).max()))


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 64), (1, 4096), (4, 8192), (3, 1000), (7, 2880), (2, 5121), (1, 16384), (300, 512), (2, 65536),
          (1, 70000), (33, 24)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_plain(awq, shape, dtype):
    d = inputs(*shape, dtype, seed=shape[1])
    check(awq.awq_residual_norm(**d), d, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["none", "channel", "row"])
@pytest.mark.parametrize("post", [False, True])
def test_forms(awq, dtype, kind, gate, post):
    for W, pad in ((1000, 0), (1000, 8), (333, 1), (4096, 0)):
        d = inputs(5, W, dtype, seed=3, post=post, gate=gate, kind=kind, bias=kind == "layer", pad=pad)
        check(awq.awq_residual_norm(**d, scale=0.25, eps=1e-5), d, dtype, scale=0.25, eps=1e-5)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_parts_left_out(awq, dtype):
    for kw in (dict(residual=False), dict(weight=False), dict(residual=False, weight=False, post=True, gate="channel"),
               dict(weight=False, post=True, bias=True, kind="layer")):
        for W in (640, 77):
            d = inputs(4, W, dtype, seed=5, **kw)
            check(awq.awq_residual_norm(**d, scale=-1.5), d, dtype, scale=-1.5)


def test_large_mean(awq):
    # a mean far above the spread: the variance is of centred values
    d = inputs(3, 2048, "fp16", seed=6, kind="layer", residual=False, mean=300.0)
    check(awq.awq_residual_norm(**d), d, "fp16")


def test_in_place(awq):
    d = inputs(9, 1024, "bf16", seed=7, post=True)
    want = awq.awq_residual_norm(**d)
    got = awq.awq_residual_norm(**d, out=(d["residual"], d["x"]))
    assert got[0].data_ptr() == d["residual"].data_ptr() and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for W in (75, 1024):
        d = inputs(9, W, "fp16", seed=8)
        want = awq.awq_residual_norm(**d)
        awq.awq_residual_norm(**d, out=(d["residual"], d["x"]))
        assert torch.equal(d["residual"], want[0]) and torch.equal(d["x"], want[1])


def test_rows_without_content_and_not_finite(awq):
    d = inputs(4, 512, "fp16", seed=9, residual=False)
    d["x"][0] = 0
    d["x"][1, 5] = float("inf")
    d["x"][2, 7] = float("nan")
    h, y = awq.awq_residual_norm(**d)
    assert (y[0] == 0).all() and torch.isnan(y[2]).all() and torch.isfinite(y[3]).all()
    assert torch.isnan(y[1, 5]) and (y[1, :5] == 0).all()  # inf over inf, and finite over inf
    d = inputs(2, 64, "bf16", seed=10, residual=False)
    d["x"][0] = 2.0 ** 70  # squares beyond fp32: finite over inf
    assert (awq.awq_residual_norm(**d)[1][0] == 0).all()


def test_many_rows_and_graph(awq):
    d = inputs(5000, 640, "bf16", seed=11, gate="row", post=True)
    want = awq.awq_residual_norm(**d)
    check((want[0][::499], want[1][::499]), {k: v[::499] if torch.is_tensor(v) and v.dim() == 2 else v for k, v in d.items()}, "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = awq.awq_residual_norm(**d)
    d["x"].copy_(d["x"].flip(0))
    d["residual"].copy_(d["residual"].flip(0))
    d["gate"].copy_(d["gate"].flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0].flip(0)) and torch.equal(out[1], want[1].flip(0))


def test_refusals(awq):
    d = inputs(4, 64, "fp16", seed=1)
    with pytest.raises(ValueError):
        awq.awq_residual_norm(**{**d, "kind": "batch"})
    with pytest.raises(TypeError):
        awq.awq_residual_norm(**{**d, "x": d["x"].float()})
    with pytest.raises(TypeError):
        awq.awq_residual_norm(**{**d, "residual": d["residual"].bfloat16()})
    with pytest.raises(ValueError):
        awq.awq_residual_norm(**{**d, "weight": d["weight"][:32]})
    with pytest.raises(ValueError):
        awq.awq_residual_norm(**{**d, "x": d["x"].t()})
    with pytest.raises(awq.AwqError):
        awq.awq_residual_norm(**d, eps=-1.0)
    with pytest.raises(awq.AwqError):
        awq.awq_residual_norm(d["x"], post_bias=d["weight"])
    wide = torch.zeros((4, 128), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):  # in place needs dense rows
        awq.awq_residual_norm(d["x"], wide[:, :64], out=(wide[:, :64], None))
    with pytest.raises(ValueError):
        awq.awq_residual_norm(d["x"].cpu(), d["residual"])
