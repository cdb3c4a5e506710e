"""awq_moe_layer where a warp goes through many blocks of K and a block through many units: stages of a ring used again,
loads that run on into the next unit, tiles of columns added up by the block that is last with several, half tiles at
the end of H, groups across blocks of K.

Tolerance as in test_gpu_moe_layer, but for the inner activations, which are two elements' sums: the result's
rounding; u^2 of an activation, fp16 2^-25 where its second element is below the normal range, carried through
the second product; and fp32 sums (relative error 2^-23 per step of a group, of the groups and of the parts) of
products whose codes may carry an offset of 128 (bf16).  With weights of either sign that bound comes near the result
for many rows of K, so each case runs a second time without cancellation: positive inputs, zeros of 0, and codes
that are one for 64 rows of a column, so that a block of rows that is lost, taken twice or taken for another moves
the result by about its share, 64 / K.  That the tolerance is below that is asserted."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
U = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
ORDER = (0, 2, 4, 6, 1, 3, 5, 7)


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


def linear(g, E, K, N, group, dtype):
    word = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, generator=g, device="cuda", dtype=torch.int64).int()  # noqa: E731
    scales = (torch.rand((E, K // group, N), generator=g, device="cuda") * 0.2 + 0.05) / K ** 0.5
    return word(E, K, N // 8), word(E, K // group, N // 8), scales.to(DT[dtype])


def positive(g, E, K, N, group, dtype, mean):
    """A linear whose outputs of inputs near 1 are near `mean`; one code for 64 rows of a column."""
    blocks = torch.randint(-2 ** 31, 2 ** 31, (E, -(-K // 64), N // 8), generator=g, device="cuda", dtype=torch.int64).int()
    scales = (torch.rand((E, K // group, N), generator=g, device="cuda") * 0.2 + 0.9) * (mean / 7.5 / K)
    zeros = torch.zeros((E, K // group, N // 8), dtype=torch.int32, device="cuda")
    return blocks.repeat_interleave(64, 1)[:, :K].contiguous(), zeros, scales.to(DT[dtype])


def inputs(T, k, E, H, I, group, dtype, seed, base=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = dict(x=torch.randn((T, H), generator=g, device="cuda").to(DT[dtype]), weights=torch.rand((T, k), generator=g, device="cuda"),
             experts=torch.rand((T, E), generator=g, device="cuda").argsort(-1)[:, :k].int().contiguous(),
             up=linear(g, E, H, 2 * I, group, dtype), down=linear(g, E, I, H, group, dtype), group_size=group)
    if base:
        d["base"] = torch.randn((T, H), generator=g, device="cuda").to(DT[dtype])
    return d


def times(x, dx, w, e, group, offset, u):
    """x times the expert's matrix in 64 bits, and the bound of the error of an fp32 evaluation of x known to dx."""
    qweight, qzeros, scales = (t[e] for t in w)
    K, N = qweight.shape[0], scales.shape[1]
    matrix, size = (torch.empty((K, N), dtype=torch.float64, device="cuda") for _ in range(2))
    for i, column in enumerate(ORDER):
        c = (qweight >> 4 * i & 15).double()
        z = (qzeros >> 4 * i & 15).double().repeat_interleave(group, 0)
        s = scales[:, column::8].double().repeat_interleave(group, 0)
        matrix[:, column::8], size[:, column::8] = (c - z) * s, (c + z + 2 * offset) * s.abs()
    steps = 2.0 ** -23 * (group / 16 + K / group + 24)
    return x @ matrix, steps * (x.abs() @ size) + (dx + u * x.abs()) @ matrix.abs()


def without_signs(d, dtype, seed):
    """The same places with positive inputs and weights."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, H, I = d["up"][0].shape[0], d["x"].shape[1], d["down"][0].shape[1]
    return dict(x=(0.5 + torch.rand(d["x"].shape, generator=g, device="cuda")).to(DT[dtype]), weights=d["weights"] + 0.1,
                experts=d["experts"], up=positive(g, E, H, 2 * I, d["group_size"], dtype, 4.0),
                down=positive(g, E, I, H, d["group_size"], dtype, 0.5), group_size=d["group_size"])


def check(out, d, dtype, share=None):
    offset, u, I = 128 if dtype == "bf16" else 0, U[dtype], d["down"][0].shape[1]
    want = d["base"].double() if "base" in d else torch.zeros(d["x"].shape, dtype=torch.float64, device="cuda")
    bound = 2.0 ** -22 * want.abs()
    for e in sorted(set(d["experts"].flatten().tolist())):
        if not 0 <= e < d["up"][0].shape[0]:
            continue
        token, place = (d["experts"] == e).nonzero(as_tuple=True)
        x = d["x"][token].double()
        both, near = times(x, torch.zeros_like(x), d["up"], e, d["group_size"], offset, 0.0)
        (g, v), (dg, dv) = both.chunk(2, -1), near.chunk(2, -1)
        silu = g * torch.sigmoid(g)
        act = silu * v
        dact = 1.1 * v.abs() * dg + silu.abs() * dv + 1.1 * dg * dv + 2.0 ** -20 * act.abs() + (2.0 ** -25 if dtype == "fp16" else 0)
        y, dy = times(act, dact, d["down"], e, d["group_size"], offset, u * u)
        w = d["weights"][token, place].double()[:, None]
        want = want.index_add(0, token, w * y)
        bound = bound.index_add(0, token, w.abs() * (dy + 2.0 ** -21 * y.abs()))
    bound = bound + 2.0 ** -21 * d["experts"].shape[1] * want.abs()
    tol = u * want.abs() + bound * (1 + u) + (2.0 ** -24 if dtype == "fp16" else 0)
    err = (out.double() - want).abs()
    assert (err <= tol).all(), (err / tol).max()
    return want
    if share:
        assert (tol < share * want).all()


# T, k, E, H, I, group
CASES = [
    (2, 2, 3, 2112, 1600, 64),       # blocks of K that do not divide by the warps, H % 128 == 64
    (16, 8, 64, 1088, 1088, 64),     # more units than block slots in both products, half tiles
    (16, 8, 64, 1088, 1088, 32),     # two groups in a block of K
    (16, 4, 40, 1344, 1344, 192),    # groups of three blocks
    (16, 4, 40, 1344, 1344, 448),    # groups of seven, across warps
    (16, 2, 8, 2048, 4096, 128),     # several rows of an expert
    (1, 8, 16, 4096, 2048, 128),
    (3, 2, 8, 4096, 14336, 128),
    (16, 8, 128, 4096, 1792, 128),
    (1, 1, 2, 8192, 512, 128),
    (16, 32, 40, 576, 640, 64),      # all 512 places
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_layer(awq, case, dtype):
    d = inputs(*CASES[case], dtype, seed=case, base=case % 2 == 0)
    out = awq.awq_moe_layer(**d)
    check(out, d, dtype)
    for _ in range(3):
        assert torch.equal(out, awq.awq_moe_layer(**d))
    d = without_signs(d, dtype, seed=100 + case)
    K = max(CASES[case][3:5])
    # bf16 rounds to 2^-8 twice: for the longest K four blocks' share
    check(awq.awq_moe_layer(**d), d, dtype, share=64 / K if dtype == "fp16" or K <= 4096 else 256 / K)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", [0, 1, 5, 8])
def test_errors_are_the_results_rounding(awq, case, dtype):
    # Nothing else is rounded to the element type: fp32 errors and u^2 of the activations are below a hundredth of u, and
    # an activation of one element alone would add as much as the result's rounding, a root mean square of 1.41 times it.
    d = inputs(*CASES[case], dtype, seed=60 + case, base=False)
    out = awq.awq_moe_layer(**d)
    want = check(out, d, dtype)
    rms = lambda x: x.square().mean().sqrt()  # noqa: E731
    assert rms(out.double() - want) <= 1.1 * rms(want.to(DT[dtype]).double() - want)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_places_left_out_and_repeated(awq, dtype):
    d = inputs(16, 8, 40, 1088, 1088, 64, dtype, seed=30)
    d["experts"][3] = -1
    d["experts"][5, ::2] = 40
    d["experts"][7] = 11
    d["experts"][8:12, 2] = 11
    out = awq.awq_moe_layer(**d)
    check(out, d, dtype)
    assert torch.equal(out[3], d["base"][3])


@pytest.mark.parametrize("size", [0, 1, 8])
def test_waits_that_give_up(awq, size):
    # as if no copy arrived in time: an error status, tensors around the outputs as they were, and the next call is right
    d = inputs(*CASES[size], "bf16", seed=31, base=False)
    T, H = d["x"].shape
    around = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
    need = awq.awq_moe_layer_workspace_size(T, d["experts"].shape[1], H, d["down"][0].shape[1])
    ws = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
    awq.selftest_attention_give_up(True)
    try:
        awq.awq_moe_layer(**d, out=around[1:-1], workspace=ws[256:256 + need])
    finally:
        awq.selftest_attention_give_up(False)
    with pytest.raises(awq.AwqError):
        awq.device_status()
    assert (around[0] == 7).all() and (around[-1] == 7).all() and (ws[:256] == 7).all() and (ws[256 + need:] == 7).all()
    check(awq.awq_moe_layer(**d, workspace=ws[256:256 + need]), d, "bf16")
