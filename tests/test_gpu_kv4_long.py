"""awq_attention_kv4 where every warp goes through many tiles: copies that reuse a ring's stages, pages looked up batch
by batch, units and parts that begin and end anywhere, for every head size and number of query rows.

Every key counts (scale 0): all probabilities are equal, the values +1 or -1 at random, so the result is a mean in
which a tile of 16 keys that is lost or taken twice stands out by some 4 / N.  Keys of weight 1, factors that fp16
holds exactly, sums of whole numbers: what rounds is a run's sum of tiles (each addition 2^-23 of it; a warp has fewer
than 100 tiles), the quotients and sums of its parts (16 steps), and the result, u |y| (u = 2^-11 fp16, 2^-8 bf16).
That the tolerance is below a lost tile is asserted.

Logits as usual: sampled sequences in 64 bits, with the tolerances of test_gpu_kv4_factors."""
import numpy as np
import pytest
import torch

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


def quantized(x, group):
    """(code * scale, minimum, scale) in 64 bits of x [..., D], by the definition."""
    by = x.float().unflatten(-1, (-1, group))
    low, high = by.amin(-1, keepdim=True), by.amax(-1, keepdim=True)
    scale = ((high * 0.5 - low * 0.5) / 7.5).to(x.dtype).float()
    code = torch.round((by * 0.5 - low * 0.5) / (scale * 0.5)).clamp(0, 15)
    wide = lambda t: t.double().expand_as(by).flatten(-2)  # noqa: E731
    return code.double().mul(scale.double()).flatten(-2), wide(low), wide(scale)


def make(awq, B, n, hq, hkv, D, group, lens, page, dtype, seed, signs=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = -(-max(lens) // page)
    total = B * per + 1
    pages = torch.randperm(total, generator=g, device="cuda")[:B * per].view(B, per).int()
    cache = torch.full((total, hkv, awq.awq_kv4_page_bytes(page, D, group)), 255, dtype=torch.uint8, device="cuda")
    keys, values = [], []
    for b in range(B):
        k = torch.randn((lens[b], hkv, D), generator=g, device="cuda").to(DT[dtype])
        if signs:
            v = torch.randint(0, 2, (lens[b], hkv, D), generator=g, device="cuda", dtype=torch.int64).mul(2).sub(1).to(DT[dtype])
            v[..., ::group], v[..., 1::group] = 1, -1  # a group's extremes, whatever the others are
        else:
            v = torch.randn((lens[b], hkv, D), generator=g, device="cuda").to(DT[dtype])
        at = torch.arange(lens[b], device="cuda")
        if lens[b]:
            awq.awq_rope_append_kv4(None, k, v, None, None, cache, (pages[b, at // page] * page + at % page).int(), group_size=group)
        keys.append(k)
        values.append(v)
    q = torch.randn((B, n, hq, D), generator=g, device="cuda").to(DT[dtype])
    call = dict(q=q, cache=cache, pages=pages, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), group_size=group)
    return call, keys, values


def ragged(B, top):
    lens = [max(1, top - (top * (7 * i % B)) // (2 * B) - 5 * i % 97) for i in range(B)]
    lens[B // 2] = 0
    return lens


# B, n, hq, hkv, D, group, longest, page, window, sinks, tiles of the call at least
CASES = [
    (48, 1, 32, 8, 64, 64, 5500, 16, 0, 0, 80000),
    (32, 4, 24, 4, 64, 32, 4000, 48, 0, 0, 40000),         # 24 rows of a head
    (32, 1, 8, 8, 96, 32, 7500, 32, 0, 0, 80000),
    (64, 1, 24, 2, 96, 32, 7000, 16, 0, 0, 40000),         # 12 rows
    (48, 1, 64, 8, 128, 128, 5500, 16, 0, 0, 80000),
    (48, 1, 64, 8, 128, 64, 5500, 64, 0, 0, 80000),
    (48, 1, 16, 8, 128, 32, 5500, 16, 0, 0, 80000),
    (24, 2, 40, 4, 128, 128, 5000, 16, 0, 0, 40000),       # 20 rows
    (24, 2, 24, 4, 128, 32, 9500, 128, 0, 0, 40000),       # 12 rows
    (32, 1, 16, 4, 256, 64, 7000, 16, 0, 0, 40000),
    (48, 5, 6, 2, 256, 128, 5000, 16, 0, 0, 40000),        # 15 rows
    (24, 1, 32, 8, 256, 32, 4700, 16, 0, 0, 40000),
    (48, 1, 32, 8, 128, 128, 9000, 16, 4500, 40, 80000),   # windows
    (48, 3, 8, 8, 64, 32, 9000, 32, 4500, 100, 80000),
    (40, 1, 24, 8, 96, 32, 9001, 32, 1024, 4, 19000),
    (300, 1, 32, 8, 128, 128, 900, 16, 0, 0, 80000),       # more sequences than entries of a block's table
    (1, 1, 8, 2, 128, 128, 100000, 64, 0, 0, 12000),
    (2, 3, 12, 2, 256, 64, 60000, 16, 0, 0, 20000),
    (2, 1, 16, 1, 64, 64, 100000, 16, 0, 0, 9000),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_long(awq, case, dtype):
    B, n, hq, hkv, D, group, longest, page, window, sinks, least = CASES[case]
    lens = ragged(B, longest) if B > 2 else [longest - 77 * i for i in range(B)]
    rows = n * hq // hkv
    tile = 16 if rows > 8 and D <= 128 else 8
    seen_by_all = [min(x, window + n + sinks if window else x) for x in lens]
    assert sum(x // 16 for x in seen_by_all) * hkv * -(-rows // tile) >= least
    call, keys, values = make(awq, B, n, hq, hkv, D, group, lens, page, dtype, seed=case)
    out = awq.awq_attention_kv4(**call, window=window, sinks=sinks, scale=0.0)
    usual = awq.awq_attention_kv4(**call, window=window, sinks=sinks)
    for again, kw in ((out, dict(scale=0.0)), (usual, {})):
        assert torch.equal(again, awq.awq_attention_kv4(**call, window=window, sinks=sinks, **kw))
    sampled = set(range(0, B, max(1, B // 4))) | {B - 1, B // 2}
    for b in range(B):
        if lens[b] == 0:
            assert (out[b] == 0).all() and (usual[b] == 0).all()
            continue
        cs, low, scale = quantized(values[b], group)
        v = cs + low
        total = torch.cat([torch.zeros_like(v[:1]), v.cumsum(0)])
        if b in sampled:
            kc, km, _ = quantized(keys[b], group)
        for i in range(n):
            at = lens[b] - n + i
            if at < 0:
                assert (out[b, i] == 0).all() and (usual[b, i] == 0).all()
                continue
            first = max(0, at - window + 1) if window else 0
            few = min(first, sinks)
            N = at + 1 - first + few
            want = (total[at + 1] - total[first] + total[few]) / N  # [hkv, D]
            got = out[b, i].double().view(hkv, -1, D)
            # sums of s |c - 8| and |m + 8 s|, 16 s / 2 and 1 at most for values of +1 and -1
            tol = U[dtype] * want.abs() + 2.0 ** -22 * 116 * 2.01
            assert ((got - want[:, None]).abs() <= tol[:, None]).all(), (b, i, ((got - want[:, None]).abs() / tol[:, None]).max())
            if N >= 64:
                lost = (first // 16 + 1 + (at // 16 - first // 16 - 1) // 2) * 16  # some whole tile of those seen
                without = (want * N - total[lost + 16] + total[lost]) / (N - 16)
                assert ((without - want).abs() > tol).any()
            if b not in sampled:
                continue
            keep = torch.cat([torch.arange(few), torch.arange(first, at + 1)]).cuda()
            q = call["q"][b, i].double().view(hkv, -1, D)
            z = torch.einsum("hgd,jhd->hgj", q, (kc + km)[keep]) / D ** 0.5
            Z = torch.einsum("hgd,jhd->hgj", q.abs(), (kc + km.abs())[keep]) / D ** 0.5
            p = torch.softmax(z, dim=-1)
            moved = 2.0 ** -23 * ((D + 16) * Z + 2 * z.abs() + 2 * z.abs().amax(-1, keepdim=True))
            if dtype == "bf16":
                moved = moved + 2.0 ** -29 / D ** 0.5 * q.abs().amax(-1, keepdim=True) * kc[keep].sum(-1).t()[:, None]
            moved = moved * p
            mean = lambda w, x: torch.einsum("hgj,jhd->hgd", w, x[keep])  # noqa: E731
            y, S, M = mean(p, v), mean(p, (cs - 8 * scale).abs()), mean(p, (low + 8 * scale).abs())
            heaviest = torch.stack([(p[h, :, :, None] * scale[keep, h][None]).amax(1) for h in range(hkv)])  # [hkv, rows, D]
            tol = U[dtype] * y.abs() + (2.0 ** -11 if dtype == "bf16" else 2.0 ** -22) * S + mean(moved, (cs - 8 * scale).abs() + (low + 8 * scale).abs()) \
                + (moved.sum(-1, keepdim=True) + 2.0 ** -22 * (N / 16 + 64)) * (S + M) + N * 15 * 2.0 ** -32 * heaviest + 2.0 ** -25
            err = (usual[b, i].double().view(hkv, -1, D) - y).abs()
            assert (err <= tol).all(), (b, i, (err / tol).max())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B,hq,hkv,D,group,longest", [(4, 64, 8, 128, 64, 60000), (7, 64, 8, 128, 128, 24000), (1, 40, 8, 64, 32, 100000),
                                                      (2, 24, 2, 96, 32, 40000), (8, 40, 8, 256, 64, 12000)])
def test_sums_do_not_drift(awq, B, hq, hkv, D, group, longest, dtype):
    # A result over many keys is a small mean of values of either sign.  Tensor cores cut a sum's last bits off where they add
    # to it: a sum that grows along a warp's keys leaves all results off to one side.  The mean of the errors is free of the
    # results' own rounding (five times its spread over the mean's root is left for it).  Sums of both signs lose on both
    # sides: 2^-19, half a step of 2^-21 of eight terms of the values' size, 1, is left for what they keep to one side, and
    # 2^-20 for exponentials and fp32 sums, which round to nearest.
    lens = [longest - 1001 * i for i in range(B)]
    call, keys, values = make(awq, B, 1, hq, hkv, D, group, lens, 16, dtype, seed=D, signs=False)
    out = awq.awq_attention_kv4(**call)
    errors, sizes = [], []
    for b in range(B):
        (kc, km, _), (cs, low, _) = quantized(keys[b], group), quantized(values[b], group)
        q = call["q"][b, 0].double().view(hkv, -1, D)
        p = torch.softmax(torch.einsum("hgd,jhd->hgj", q, kc + km) / D ** 0.5, dim=-1)
        want = torch.einsum("hgj,jhd->hgd", p, cs + low)
        errors.append((out[b, 0].double().view(hkv, -1, D) - want).flatten())
        sizes.append(want.flatten())
    error, size = torch.cat(errors), torch.cat(sizes)
    spread = U[dtype] * size.square().mean().sqrt()
    assert abs(error.mean()) <= 2.0 ** -19 + 2.0 ** -20 + 5 * spread / len(error) ** 0.5, error.mean()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,group,hq,hkv", [(64, 64, 8, 2), (96, 32, 6, 2), (128, 128, 8, 2), (128, 64, 24, 2), (256, 64, 8, 2)])
def test_every_key_of_a_window_counts(awq, D, group, hq, hkv, dtype):
    # one key more or less at an edge of the window or the first tokens moves the mean by 1 / N: more than the tolerance
    n, lens = 3, [700, 1500, 65, 130, 3100, 2]
    call, _, values = make(awq, len(lens), n, hq, hkv, D, group, lens, 16, dtype, seed=D)
    for window, sinks in ((1, 0), (1, 1), (7, 0), (16, 16), (17, 15), (33, 40), (64, 1), (100, 129), (640, 3), (0, 0)):
        out = awq.awq_attention_kv4(**call, window=window, sinks=sinks, scale=0.0).double().view(len(lens), n, hkv, -1, D)
        for b, count in enumerate(lens):
            cs, low, _ = quantized(values[b], group)
            for i in range(n):
                at = count - n + i
                if at < 0:
                    assert (out[b, i] == 0).all()
                    continue
                keep = torch.tensor([j for j in range(at + 1) if window == 0 or j > at - window or j < sinks], device="cuda")
                want = (cs + low)[keep].mean(0)
                tol = U[dtype] * want.abs() + 2.0 ** -22 * 116 * 2.01
                assert ((out[b, i] - want[:, None]).abs() <= tol[:, None]).all(), (window, sinks, b, i)
                if 2 <= len(keep) <= 1000:
                    without = (cs + low)[keep[1:]].mean(0)
                    assert ((without - want).abs() > tol).any()
