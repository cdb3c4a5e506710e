"""awq_attention_kv4 where keys' values differ in size by many powers of two: the factor of a value, probability
times scale, is held in fp16 relative to the largest of its own query row and group of elements, so neither keys
that the row does not see, nor seen ones of no weight, nor other groups take bits from it.

Tolerance, per element of a group, y = sum_j p_j s_j (c_j - 8) + p_j (m_j + 8 s_j) over N keys, S = sum_j p_j s_j |c_j - 8|,
M = sum_j p_j |m_j + 8 s_j|:
  the result's rounding u |y| (u = 2^-11 fp16, 2^-8 bf16; below fp16's normal range half of 2^-24);
  the factor's: 2^-11 S (bf16, one fp16 term), 2^-22 S (fp16, two terms), and below fp16's normal range 2^-25 of a
  factor where the largest p s of the row and group is 2^7 or more: N * 15 * 2^-32 * max_j p_j s_j;
  fp32: a logit is a sum of D products, each addition at most 2^-23 of Z_j = |scale| sum |q| (c s + |m|), with the
  parameters' and the exponential's 16 steps more, and its distance to the row's largest; bf16 queries become fp16
  numbers of which the row's largest is 2^4 or more: 2^-25 * 2^-4 of it per element.  A logit's error moves its p_j by
  as much, and the sum of all p likewise.  Sums over N keys in tiles of 16: 2^-22 (N / 16 + 64)."""
import math

import numpy as np
import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
U = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
HUGE = {"fp16": 6e4, "bf16": 1e30}


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


def on_device(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype]).cuda()


def call(awq, q, k, v, group, dtype, page=16, **kw):
    """One sequence's keys and values [tokens, heads, D], queries [n, Hq, D] (numpy): the call's output."""
    tokens, heads, D = k.shape
    pages = torch.randperm(-(-tokens // page) + 1, generator=torch.Generator().manual_seed(1))[1:].int()
    at = torch.arange(tokens)
    cache = torch.full((len(pages) + 1, heads, awq.awq_kv4_page_bytes(page, D, group)), 255, dtype=torch.uint8, device="cuda")
    awq.awq_rope_append_kv4(None, on_device(k, dtype), on_device(v, dtype), None, None, cache,
                            (pages[at // page] * page + at % page).int().cuda(), group_size=group)
    return awq.awq_attention_kv4(on_device(q, dtype)[None], cache, pages[None].cuda(),
                                 torch.tensor([tokens], dtype=torch.int32, device="cuda"), group_size=group, **kw)[0]


def plain(q, k, v, group, dtype, scale=None, window=0, sinks=0):
    """(the 64-bit result [n, Hq, D], its tolerance) of the same."""
    elements = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype]).float().numpy()  # noqa: E731
    q = elements(q).astype(np.float64)
    n, Hq, D = q.shape
    tokens, heads, _ = k.shape
    scale = 1 / math.sqrt(D) if scale is None else scale
    parts = []
    for x in (k, v):
        code, s, m = (a.astype(np.float64) for a in step.quantize(elements(x), group, dtype))
        s, m = np.repeat(s, group, -1), np.repeat(m, group, -1)
        parts.append((code * s, m, s))
    (kc, km, _), (vc, vm, vs) = parts
    eight = 8 * vs
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for i in range(n):
        at = tokens - n + i
        seen = np.array([j for j in range(at + 1) if window == 0 or j > at - window or j < sinks])
        N = len(seen)
        for h in range(Hq):
            hk, row = h // (Hq // heads), q[i, h]
            z = scale * ((kc + km)[seen, hk] @ row)
            Z = abs(scale) * ((kc + np.abs(km))[seen, hk] @ np.abs(row))
            p = np.exp(z - z.max())
            p /= p.sum()
            y, S, M = (p @ a[seen, hk] for a in (vc + vm, np.abs(vc - eight), np.abs(vm + eight)))
            moved = 2.0 ** -23 * ((D + 16) * Z + 2 * np.abs(z) + 2 * np.abs(z).max())
            if dtype == "bf16":
                moved += 2.0 ** -29 * np.abs(row).max() * abs(scale) * kc[seen, hk].sum(-1)
            moved *= p
            out[i, h] = y
            tol[i, h] = U[dtype] * np.abs(y) + (2.0 ** -11 if dtype == "bf16" else 2.0 ** -22) * S \
                + moved @ (np.abs(vc - eight) + np.abs(vm + eight))[seen, hk] + (moved.sum() + 2.0 ** -22 * (N / 16 + 64)) * (S + M) \
                + N * 15 * 2.0 ** -32 * (p[:, None] * vs[seen, hk]).max(0) + (2.0 ** -25 if dtype == "fp16" else 0)
    return out, tol


def check(got, want, tol, where=...):
    got = got.double().cpu().numpy()
    assert np.isfinite(got[where]).all()
    worst = (np.abs(got - want) / tol)[where].max()
    assert worst <= 1, worst


# D, group, query heads, key/value heads: up to 8 rows of a head and more, every head size
SHAPES = [(64, 32, 2, 1), (64, 64, 8, 1), (96, 32, 2, 1), (128, 128, 2, 1), (128, 64, 2, 2), (128, 32, 4, 1), (128, 128, 16, 2),
          (256, 128, 2, 1), (256, 32, 6, 1)]


def draw(D, hq, hkv, n, tokens, seed):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((n, hq, D)), rng.standard_normal((tokens, hkv, D)), rng.standard_normal((tokens, hkv, D))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("tokens", [40, 700, 3000])
@pytest.mark.parametrize("shape", SHAPES)
def test_a_newer_token_of_huge_values(awq, shape, tokens, dtype):
    D, group, hq, hkv = shape
    q, k, v = draw(D, hq, hkv, 4, tokens, seed=D + tokens)
    good = call(awq, q, k, v, group, dtype)
    v[-1] *= HUGE[dtype] / np.abs(v[-1]).max()  # seen by the last of the four alone
    got = call(awq, q, k, v, group, dtype)
    want, tol = plain(q, k, v, group, dtype)
    check(got, want, tol)
    assert torch.equal(got[:3], good[:3])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES[::2])
def test_a_token_of_huge_values_that_leaves_the_window(awq, shape, dtype):
    D, group, hq, hkv = shape
    q, k, v = draw(D, hq, hkv, 4, 90, seed=D)
    good = call(awq, q, k, v, group, dtype, window=30, sinks=2)
    v[90 - 4 - 30 + 1] *= HUGE[dtype] / np.abs(v[57]).max()  # the last key of the first new token's window
    got = call(awq, q, k, v, group, dtype, window=30, sinks=2)
    want, tol = plain(q, k, v, group, dtype, window=30, sinks=2)
    check(got, want, tol)
    assert torch.equal(got[1:], good[1:])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("where", [0, 33, 639, 1999])
@pytest.mark.parametrize("shape", SHAPES)
def test_a_key_of_no_weight_with_huge_values(awq, shape, where, dtype):
    # its logit is at least 100 (bf16) or 40 (fp16) below the others' in every row but the last query head's, which singles it out
    D, group, hq, hkv = shape
    q, k, v = draw(D, hq, hkv, 1, 2000, seed=where)
    q[:, :, 0] = np.abs(q[:, :, 0]) + 2
    q[:, -1, 0] *= -1
    k[where, :, 0] = -50.0 * math.sqrt(D) if dtype == "bf16" else -20.0 * math.sqrt(D)
    v[where] *= HUGE[dtype] / np.abs(v[where]).max()
    want, tol = plain(q, k, v, group, dtype)
    got = call(awq, q, k, v, group, dtype)
    check(got, want, tol)
    assert np.abs(want[:, 0]).max() < 2 and np.abs(want[:, -1]).max() > 1e3


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("shape", SHAPES)
def test_sizes_that_grow_and_shrink_along_the_keys(awq, shape, order, dtype):
    # values by 2^-14 (fp16) or 2^-60 (bf16) to as much above along the keys, weights against them
    D, group, hq, hkv = shape
    q, k, v = draw(D, hq, hkv, 2, 900, seed=7)
    reach = 14 if dtype == "fp16" else 60
    size = np.linspace(-reach, reach, 900)[::order, None]
    v = v * 2.0 ** np.minimum(size, 12 if dtype == "fp16" else 60)[..., None]
    q[:, :, 0] = math.sqrt(D) * np.linspace(0.2, 1.0, 2 * hq).reshape(2, hq)
    k[:, :, 0] = -0.7 * size  # logits by -0.7 r size: the larger the value, the smaller its weight
    want, tol = plain(q, k, v, group, dtype)
    check(call(awq, q, k, v, group, dtype), want, tol)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] > s[1]])
def test_groups_of_different_sizes(awq, shape, dtype):
    D, group, hq, hkv = shape
    q, k, v = draw(D, hq, hkv, 2, 500, seed=9)
    groups = D // group
    sizes = np.linspace(10, -12, groups) if dtype == "fp16" else np.linspace(40, -80, groups)
    v = v * np.repeat(2.0 ** sizes, group)
    want, tol = plain(q, k, v, group, dtype)
    check(call(awq, q, k, v, group, dtype), want, tol)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_smallest_and_largest_values(awq, dtype):
    # down to the type's smallest normal numbers; bf16 up to 2^100, above which products may overflow
    for size in ((2.0 ** -13, 2.0 ** 13) if dtype == "fp16" else (2.0 ** -100, 2.0 ** 97)):
        q, k, v = draw(128, 4, 1, 2, 300, seed=4)
        v = v * size
        want, tol = plain(q, k, v, 64, dtype)
        check(call(awq, q, k, v, 64, dtype), want, tol)


def test_keys_and_queries_of_any_size_bf16(awq):
    # products near 1 of keys of 2^90 and queries of 2^-90, and the other way round
    for size in (2.0 ** 90, 2.0 ** -90):
        q, k, v = draw(128, 4, 1, 2, 300, seed=5)
        q, k = q / size, k * size
        want, tol = plain(q, k, v, 64, "bf16")
        check(call(awq, q, k, v, 64, "bf16"), want, tol)
