"""Forms of the calls around a 4-bit cache that give what the plain form of the call gives: in place, of odd strides and
addresses, of broadcast inputs, two captured calls side by side, a million tokens, every place at one expert."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


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


def shifted(x, by=1):
    """The same numbers `by` elements off, in rows by `by` longer."""
    wide = torch.zeros((*x.shape[:-1], x.shape[-1] + 2 * by), dtype=x.dtype, device=x.device)
    view = wide[..., by:-by]
    view.copy_(x)
    return view


# tokens, query heads, key/value heads, head size, group, rotated, pairs side by side
APPEND = [(5, 8, 2, 128, 128, 128, False), (7, 6, 2, 96, 32, 96, True), (33, 4, 4, 128, 32, 64, True), (19, 14, 2, 256, 64, 256, False),
          (40, 3, 3, 64, 32, 30, False), (6, 2, 1, 256, 128, 250, True), (300, 40, 40, 96, 32, 96, False), (2, 70, 1, 64, 64, 64, False)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_in_place_and_of_odd_strides(awq, case, dtype):
    T, hq, hkv, D, group, rot, interleaved = APPEND[case]
    g = torch.Generator(device="cuda").manual_seed(case)
    q, k, v = (torch.randn((T, h, D), generator=g, device="cuda").to(dtype) for h in (hq, hkv, hkv))
    table, pos = awq.awq_rope_table(512, rot), torch.arange(T, dtype=torch.int32, device="cuda") + 3
    slots = torch.randperm(T + 13, generator=g, device="cuda")[:T].int()
    new = lambda: torch.zeros((-(-(T + 13) // 16), hkv, awq.awq_kv4_page_bytes(16, D, group)), dtype=torch.uint8, device="cuda")  # noqa: E731
    cache = new()
    call = dict(positions=pos, table=table, slots=slots, group_size=group, interleaved=interleaved)
    want = awq.awq_rope_append_kv4(q, k, v, cache=cache, **call)
    for views in ((q.clone(), k, v), (shifted(q), shifted(k), shifted(v)), (shifted(q, 8), k, shifted(v, 8)), (q.clone(), shifted(k, 3), v)):
        for in_place in (False, True):
            again, qv = new(), shifted(views[0]) if views[0].stride(1) % 8 else views[0].clone()
            got = awq.awq_rope_append_kv4(qv, views[1], views[2], cache=again, q_out=qv if in_place else None, **call)
            assert torch.equal(got, want) and torch.equal(again, cache) and (got.data_ptr() == qv.data_ptr()) == in_place
    k0, v0 = awq.awq_kv4_read(cache, slots, D, group_size=group, dtype=dtype)
    flat = torch.zeros((2 * T * hkv * D + 2,), dtype=dtype, device="cuda")  # outputs off a vector
    out = flat[1:1 + T * hkv * D].view(T, hkv, D), flat[1 + T * hkv * D:-1].view(T, hkv, D)
    got = awq.awq_kv4_read(cache, slots, D, group_size=group, dtype=dtype, out=out)
    assert got[0].data_ptr() == out[0].data_ptr() and torch.equal(got[0], k0) and torch.equal(got[1], v0)
    assert flat[0] == 0 and flat[-1] == 0


def attention_inputs(awq, lens, hq, hkv, D, group, n=1, dtype=torch.float16, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = -(-max(lens) // 16)
    pages = torch.randperm(len(lens) * per, generator=g, device="cuda").view(len(lens), per).int()
    cache = torch.full((len(lens) * per, hkv, awq.awq_kv4_page_bytes(16, D, group)), 255, dtype=torch.uint8, device="cuda")
    for b, count in enumerate(lens):
        at = torch.arange(count, device="cuda")
        k, v = (torch.randn((count, hkv, D), generator=g, device="cuda").to(dtype) for _ in range(2))
        awq.awq_rope_append_kv4(None, k, v, None, None, cache, (pages[b, at // 16] * 16 + at % 16).int(), group_size=group)
    q = torch.randn((len(lens), n, hq, D), generator=g, device="cuda").to(dtype)
    return dict(q=q, cache=cache, pages=pages, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), group_size=group)


def test_attention_of_broadcast_queries_and_tables(awq):
    call = attention_inputs(awq, [700, 700, 700], 8, 2, 128, 64, n=2)
    call["pages"] = call["pages"][:1].expand(3, -1)  # one sequence's pages for all: stride 0
    for q in (call["q"][:1].expand(3, -1, -1, -1), call["q"][:, :1].expand(-1, 2, -1, -1), call["q"][:, :, :1].expand(-1, -1, 8, -1)):
        got, want = (awq.awq_attention_kv4(**{**call, "q": t}) for t in (q, q.contiguous()))
        assert torch.equal(got, want)
    one = awq.awq_attention_kv4(**{**call, "q": call["q"][:1].expand(3, -1, -1, -1)})
    # the sequences are alike, but cut at other keys: equal to their rounding
    assert (one - one[:1]).abs().max() <= 2 * 2.0 ** -11 * one.abs().max()


def test_captured_calls_side_by_side(awq):
    # two graphs with workspaces of their own, replayed at a time on two streams, beside eager calls on a third
    calls = [attention_inputs(awq, lens, 16, 4, 128, 128, seed=s) for s, lens in enumerate(([5000, 30, 900], [40, 7000], [3000]))]
    want = [awq.awq_attention_kv4(**c) for c in calls]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(3)]
    for c in calls[:2]:
        ws = torch.empty((awq.awq_attention_kv4_workspace_size(len(c["lens"]), 1, 16, 4, 128),), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(awq.awq_attention_kv4(**c, workspace=ws))
        graphs.append((g, ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        with torch.cuda.stream(streams[2]):
            third = awq.awq_attention_kv4(**calls[2])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(third, want[2])


@pytest.mark.parametrize("window,sinks", [(0, 0), (600_000, 50), (100, 7)])
def test_a_million_tokens(awq, window, sinks):
    # equal probabilities: the mean of the values that the last two tokens see
    count, hkv, D = 1_000_003, 2, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    cache = torch.zeros((-(-count // 16), hkv, awq.awq_kv4_page_bytes(16, D, 64)), dtype=torch.uint8, device="cuda")
    slots = torch.arange(count, dtype=torch.int32, device="cuda")
    k = torch.randn((count, hkv, D), generator=g, device="cuda").half()
    v = (torch.randn((count, hkv, D), generator=g, device="cuda") + torch.linspace(-1, 1, count, device="cuda")[:, None, None]).half()
    awq.awq_rope_append_kv4(None, k, v, None, None, cache, slots, group_size=64)
    q = torch.ones((1, 2, 4, D), dtype=torch.float16, device="cuda")
    pages, lens = torch.arange(-(-count // 16), dtype=torch.int32, device="cuda")[None], torch.tensor([count], dtype=torch.int32, device="cuda")
    out = awq.awq_attention_kv4(q, cache, pages, lens, group_size=64, window=window, sinks=sinks, scale=0.0).double()
    by = v.float().unflatten(-1, (1, 64))
    low, high = by.amin(-1, keepdim=True), by.amax(-1, keepdim=True)
    scale = ((high * 0.5 - low * 0.5) / 7.5).half().float()
    held = (torch.round((by * 0.5 - low * 0.5) / (scale * 0.5)).clamp(0, 15).double() * scale.double() + low.double()).flatten(-2)
    for i in range(2):
        at = count - 2 + i
        first = max(0, at - window + 1) if window else 0
        keep = torch.cat([held[:min(first, sinks)], held[first:at + 1]])
        want, size = keep.mean(0), keep.abs().mean(0)
        # the result's rounding, half a step below the normal range; sums over a warp's 60 tiles at most, and its parts
        tol = 2.0 ** -11 * want.abs() + 2.0 ** -25 + 2.0 ** -22 * 116 * (size + 8 * scale.mean())
        assert ((out[0, i].view(hkv, 2, D) - want[:, None]).abs() <= tol[:, None]).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_norm_forms(awq, dtype):
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    for T, W in ((6, 1000), (6, 1001), (700, 640), (3, 20000)):
        x, r, w, pw, gate = rand(T, W), rand(T, W), rand(W), rand(W), rand(W)
        for kw in (dict(), dict(post_weight=pw), dict(gate=gate), dict(post_weight=pw, gate=gate, kind="layer")):
            want = awq.awq_residual_norm(x, r, weight=w, **kw)
            a = x.clone()
            got = awq.awq_residual_norm(a, r, weight=w, **{**kw, "out": (torch.empty_like(x), a)})  # y in x
            assert torch.equal(got[0], want[0]) and torch.equal(a, want[1])
            b = r.clone()
            got = awq.awq_residual_norm(x, b, weight=w, **{**kw, "out": (b, torch.empty_like(x))})  # h in residual
            assert torch.equal(b, want[0]) and torch.equal(got[1], want[1])
            if "gate" in kw:  # a row of gates for all tokens, by stride 0 and spelled out
                for rows in (gate.expand(T, W), gate.expand(T, W).contiguous()):
                    got = awq.awq_residual_norm(x, r, weight=w, **{**kw, "gate": rows})
                    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            # one residual, one input for all tokens
            got = awq.awq_residual_norm(x[:1].expand(T, W), r[:1].expand(T, W), weight=w, **kw)
            assert all(torch.equal(p, q[:1].expand(T, W)) for p, q in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_every_place_at_one_expert(awq, dtype):
    # 512 places; weights of a power of two that add up to one give the expert's own result
    g = torch.Generator(device="cuda").manual_seed(5)
    word = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, generator=g, device="cuda", dtype=torch.int64).int()  # noqa: E731
    up, down = ((word(2, K, N // 8), word(2, K // 64, N // 8), (0.1 * torch.rand((2, K // 64, N), generator=g, device="cuda") / K ** 0.5).to(dtype))
                for K, N in ((320, 512), (256, 320)))
    x = torch.randn((16, 320), generator=g, device="cuda").to(dtype)
    one = awq.awq_moe_layer(x, torch.ones((16, 1), device="cuda"), torch.ones((16, 1), dtype=torch.int32, device="cuda"), up, down, group_size=64)
    all_ = awq.awq_moe_layer(x, torch.full((16, 32), 1 / 32, device="cuda"), torch.ones((16, 32), dtype=torch.int32, device="cuda"), up, down,
                             group_size=64)
    assert torch.equal(one, all_)
    assert np.isfinite(one.float().cpu().numpy()).all()
