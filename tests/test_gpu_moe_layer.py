"""GPU parity of awq_moe_layer against the 64-bit oracle.

Tolerance, per element: the result's rounding u |y| (u = 2^-11 fp16, 2^-8 bf16; fp16 results below the normal
range round to a multiple of 2^-24) and the oracle's bound: the rounding u of the inner activations, and
fp32 sums of products whose codes the kernels may carry with an offset of 128 (bf16: the code c as the number
128 + c, less (128 + zero) times the sum of x), relative error 2^-23 per step of a group, of the groups and
of the parts."""
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


@pytest.fixture(autouse=True)
def no_wait_gave_up(awq):
    yield
    awq.device_status()


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def linear(g, E, K, N, group, dtype):
    word = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, generator=g, dtype=torch.int64).to(torch.int32).cuda()  # noqa: E731
    scales = (torch.rand((E, K // group, N), generator=g) * 0.2 + 0.05) / K ** 0.5
    return word(E, K, N // 8), word(E, K // group, N // 8), scales.to(DT[dtype]).cuda()


def inputs(T, k, E, H, I, group, dtype, seed, base=True):
    g = torch.Generator().manual_seed(seed)
    experts = torch.rand((T, E), generator=g).argsort(-1)[:, :k].int().cuda()
    d = dict(x=torch.randn((T, H), generator=g).to(DT[dtype]).cuda(), weights=torch.rand((T, k), generator=g).cuda(), experts=experts,
             up=linear(g, E, H, 2 * I, group, dtype), down=linear(g, E, I, H, group, dtype), group_size=group)
    if base:
        d["base"] = torch.randn((T, H), generator=g).to(DT[dtype]).cuda()
    return d


def check(out, d, dtype):
    host = lambda w: [w[0].cpu().numpy(), w[1].cpu().numpy(), f64(w[2])]  # noqa: E731
    want, bound = step.moe_layer(f64(d["x"]), f64(d["weights"]), d["experts"].cpu().numpy(), host(d["up"]), host(d["down"]),
                                 d["group_size"], f64(d.get("base")), U[dtype], 128 if dtype == "bf16" else 0)
    tol = U[dtype] * np.abs(want) + bound * (1 + U[dtype]) + (2.0 ** -24 if dtype == "fp16" else 0)
    err = np.abs(f64(out) - want)
    assert (err <= tol).all(), float((err / tol).max())


# T, k, E, H, I, group
CASES = [
    (1, 1, 1, 128, 128, 128),
    (1, 2, 8, 256, 128, 128),
    (1, 8, 16, 512, 256, 64),
    (2, 2, 4, 1024, 512, 128),
    (3, 3, 5, 384, 896, 128),
    (4, 6, 8, 256, 192, 64),
    (5, 4, 60, 512, 128, 128),
    (8, 2, 3, 256, 256, 32),
    (9, 1, 2, 128, 384, 128),
    (13, 8, 9, 320, 160, 32),
    (16, 2, 4, 512, 512, 128),
    (16, 8, 32, 256, 128, 64),
    (2, 2, 3, 72, 40, 8),          # sizes off every tile
    (3, 2, 3, 200, 104, 8),
    (2, 3, 4, 48, 16, 16),
    (16, 1, 1, 256, 128, 128),     # every row at one expert
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_layer(awq, case, dtype):
    d = inputs(*CASES[case], dtype, seed=case, base=case % 2 == 0)
    out = awq.awq_moe_layer(**d)
    check(out, d, dtype)
    assert torch.equal(out, awq.awq_moe_layer(**d))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", [(256, 128, 128), (48, 24, 8)])
def test_places(awq, dtype, shape):
    # places without an expert whatever their weight, an expert twice in a token, tokens without any
    H, I, group = shape
    d = inputs(6, 4, 5, H, I, group, dtype, seed=40)
    d["experts"].copy_(torch.tensor([[-1, 2, 2, 5], [0, 0, 0, 0], [-1, -1, -1, -1], [4, 3, 1 << 30, 0], [-(1 << 31), 1, 1, 1],
                                     [2, 2, 2, 2]], dtype=torch.int32))
    d["weights"][0, 0] = float("nan")
    d["weights"][3, 2] = float("inf")
    d["weights"][1, 1] = 0.0
    d["weights"][1, 2] = -0.5
    out = awq.awq_moe_layer(**d)
    d["weights"] = torch.nan_to_num(d["weights"], nan=0.0, posinf=0.0)
    check(out, d, dtype)
    assert torch.equal(out[2], d["base"][2])


def test_many_duplicates(awq):
    # more rows at one expert than tokens
    d = inputs(16, 2, 2, 256, 128, 128, "fp16", seed=41)
    d["experts"] = torch.ones((16, 8), dtype=torch.int32, device="cuda")
    d["weights"] = torch.rand((16, 8), generator=torch.Generator().manual_seed(1)).cuda()
    check(awq.awq_moe_layer(**d), d, "fp16")


def test_rows_do_not_mix(awq):
    # a NaN in one token stays there
    d = inputs(5, 2, 3, 256, 128, 128, "bf16", seed=42)
    good = awq.awq_moe_layer(**d)
    d["x"][3, 17] = float("nan")
    out = awq.awq_moe_layer(**d)
    keep = [0, 1, 2, 4]
    assert torch.equal(out[keep], good[keep]) and torch.isnan(out[3]).all()


def test_strides_out_base_and_empty(awq):
    d = inputs(4, 2, 4, 256, 128, 128, "fp16", seed=43)
    want = awq.awq_moe_layer(**d)
    wide = torch.zeros((4, 512), dtype=torch.float16, device="cuda")
    wide[:, 96:352] = d["x"]
    got = awq.awq_moe_layer(**{**d, "x": wide[:, 96:352], "out": d["base"]})
    assert got.data_ptr() == d["base"].data_ptr() and torch.equal(got, want)
    wide = torch.zeros((4, 301), dtype=torch.float16, device="cuda")  # rows off every vector
    wide[:, 3:259] = d["x"]
    d = inputs(4, 2, 4, 256, 128, 128, "fp16", seed=43)
    check(awq.awq_moe_layer(**{**d, "x": wide[:, 3:259]}), d, "fp16")
    none = {**d, "x": d["x"][:0], "weights": d["weights"][:0], "experts": d["experts"][:0], "base": None}
    assert awq.awq_moe_layer(**none).shape == (0, 256)
    none = {**d, "weights": d["weights"][:, :0].contiguous(), "experts": d["experts"][:, :0].contiguous()}
    assert torch.equal(awq.awq_moe_layer(**none), d["base"])


def test_extreme_activations(awq):
    # gates far below and above zero: silu is 0 and the gate itself
    d = inputs(2, 1, 1, 128, 128, 128, "bf16", seed=44, base=False)
    d["x"] *= 2.0 ** 20
    out = awq.awq_moe_layer(**d)
    assert torch.isfinite(out).all()
    check(out, d, "bf16")


def test_graph_and_streams(awq):
    d = inputs(6, 4, 12, 512, 256, 128, "bf16", seed=45)
    want = awq.awq_moe_layer(**d)
    ws = torch.empty((awq.awq_moe_layer_workspace_size(6, 4, 512, 256),), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = awq.awq_moe_layer(**d, workspace=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = [awq.awq_moe_layer(**d) for _ in range(3)]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.equal(a, want) for a in again)
    d["experts"].copy_(d["experts"].flip(1))
    d["weights"].copy_(d["weights"].flip(1))
    graph.replay()
    torch.cuda.synchronize()
    check(out, d, "bf16")


def test_refusals(awq):
    d = inputs(4, 2, 4, 256, 128, 128, "fp16", seed=46)
    many = inputs(17, 2, 4, 128, 128, 128, "fp16", seed=46)
    with pytest.raises(awq.AwqError):
        awq.awq_moe_layer(**many)
    for change in (dict(x=d["x"].float()), dict(up=tuple(t.bfloat16() if t.dtype is torch.float16 else t for t in d["up"]))):
        with pytest.raises(TypeError):
            awq.awq_moe_layer(**{**d, **change})
    for change in (dict(down=tuple(t[:2] for t in d["down"])), dict(experts=d["experts"][:3]), dict(group_size=64),
                   dict(weights=d["weights"][:, :1]), dict(base=d["base"][:, :8]), dict(x=d["x"].cpu())):
        with pytest.raises(ValueError):
            awq.awq_moe_layer(**{**d, **change})
    with pytest.raises(awq.AwqError):  # out must not be x
        awq.awq_moe_layer(**{**d, "out": d["x"]})
    with pytest.raises(awq.AwqError):
        awq.awq_moe_layer(**d, workspace=torch.empty((16,), dtype=torch.uint8, device="cuda"))
