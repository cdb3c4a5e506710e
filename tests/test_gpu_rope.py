"""GPU parity of the rotary-position operators against the 64-bit oracle.

Tolerance, per element: one rounding to the element type (u |y|, u = 2^-11 fp16, 2^-8 bf16) of an
fp32 value a c - b s whose table entries carry one rounding (2^-24) and whose two products and sum
carry at most three more: 4 * 2^-24 * m (|a| + |b|), m the factor on cosines and sines.  fp16 results
below the normal range round to a multiple of 2^-24."""
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


def f64(t):
    return t.detach().cpu().double().numpy()


def close(y, x, positions, freq, dtype, interleaved, m=1.0):
    want = layer.rope(f64(x), positions, freq, m, interleaved)
    err = np.abs(f64(y) - want)
    half = len(freq)
    size = np.abs(f64(x))
    pair = np.zeros_like(size)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    pair[..., a] = pair[..., b] = size[..., a] + size[..., b]
    tol = U[dtype] * np.abs(want) + (4 * 2.0 ** -24 * m * pair) + (2.0 ** -25 if dtype == "fp16" else 0)
    assert (err <= tol * (1 + 1e-6)).all(), (err / np.maximum(tol, 1e-300)).max()
    assert np.array_equal(f64(y)[..., 2 * half:], f64(x)[..., 2 * half:])


SCALINGS = [("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
            ("yarn", dict(factor=8.0, original_max_position=256)), ("banded", dict(factor=8.0, original_max_position=512))]


@pytest.mark.parametrize("scaling,kw", SCALINGS)
@pytest.mark.parametrize("rot", [4, 64, 96])
def test_table(awq, scaling, kw, rot):
    n = 1000
    table = f64(awq.awq_rope_table(n, rot, base=50000.0, scaling=scaling, **kw))
    f = layer.rope_frequencies(rot, 50000.0, scaling, kw.get("factor", 1.0), kw.get("original_max_position", 0))
    m = 0.1 * np.log(8.0) + 1 if scaling == "yarn" else 1.0
    angle = np.arange(n)[:, None] * f[None]
    want = m * np.concatenate([np.cos(angle), np.sin(angle)], axis=1)
    # one fp32 rounding, and 64-bit frequencies that differ by a few ulp (n * 8 * 2^-53)
    assert (np.abs(table - want) <= 2.0 ** -24 * np.abs(want) + n * 2.0 ** -50).all()


def test_table_far_positions(awq):
    # angles of positions near 2^20 keep their accuracy (an fp32 product would be off by 0.03)
    table = f64(awq.awq_rope_table(1 << 20, 4, base=10000.0))
    p = np.arange((1 << 20) - 64, 1 << 20)
    assert np.abs(table[p, 0] - np.cos(p * 1.0)).max() < 1e-7 and np.abs(table[p, 3] - np.sin(p * 0.01)).max() < 1e-7


def fused(T, hq, hkv, d, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, (hq + 2 * hkv) * d + pad), generator=g).to(DT[dtype]).cuda()
    return (x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
            x[:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d)))


# (T, hq, hkv, d, rot, pad): one token, odd head sizes and rotated parts, misaligned rows, many tokens
CASES = [(1, 1, 1, 2, 2, 0), (1, 8, 8, 128, 128, 0), (5, 3, 1, 80, 20, 0), (7, 4, 2, 64, 64, 1), (33, 6, 2, 96, 48, 0),
         (9, 5, 5, 50, 34, 3), (300, 16, 4, 128, 64, 0), (64, 64, 8, 128, 128, 0), (17, 2, 1, 256, 256, 8), (3, 2, 2, 64, 8, 0)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,rot,pad", CASES)
def test_rope(awq, T, hq, hkv, d, rot, pad, interleaved, dtype):
    q, k, _ = fused(T, hq, hkv, d, dtype, 7 * T + d + rot, pad)
    table = awq.awq_rope_table(5000, rot)
    pos = np.random.default_rng(T).integers(0, 5000, T).astype(np.int32)
    qo, ko = awq.awq_rope(q, k, torch.from_numpy(pos).cuda(), table, interleaved=interleaved)
    f = layer.rope_frequencies(rot)
    close(qo, q, pos, f, dtype, interleaved)
    close(ko, k, pos, f, dtype, interleaved)


def test_rope_in_place_and_outputs(awq):
    q, k, _ = fused(21, 4, 2, 64, "bf16", 5)
    table, pos = awq.awq_rope_table(64, 64), torch.arange(21, dtype=torch.int32, device="cuda")
    want = awq.awq_rope(q, k, pos, table)
    q2, k2 = q.clone(), torch.empty_like(k, memory_format=torch.contiguous_format)
    a, b = awq.awq_rope(q2, k, pos, table, q_out=q2, k_out=k2)
    assert a is q2 and b is k2 and torch.equal(a, want[0]) and torch.equal(b, want[1])
    rows = q.untyped_storage()  # in place inside the fused rows: q's strides
    c, _ = awq.awq_rope(q, k, pos, table, q_out=q)
    assert c.untyped_storage().data_ptr() == rows.data_ptr() and torch.equal(c, want[0])
    with pytest.raises(ValueError):
        awq.awq_rope(q, k, pos, table, q_out=torch.empty((21, 4, 65), dtype=q.dtype, device="cuda")[..., :64])


def test_rope_positions_outside_the_table(awq):
    q, k, _ = fused(3, 2, 1, 64, "fp16", 6)
    table = awq.awq_rope_table(16, 32)
    qo, ko = awq.awq_rope(q, k, torch.tensor([-1, 3, 16], dtype=torch.int32, device="cuda"), table)
    for x, src in ((qo, q), (ko, k)):
        assert x[[0, 2], :, :32].isnan().all() and x[1].isfinite().all() and torch.equal(x[..., 32:], src[..., 32:])


@pytest.mark.parametrize("layout", ["page, token, head", "page, head, token", "keys and values side by side"])
@pytest.mark.parametrize("T,hq,hkv,d,rot,page", [(1, 4, 4, 64, 64, 16), (13, 8, 2, 128, 128, 20), (40, 3, 1, 96, 32, 1),
                                                 (6, 2, 2, 50, 10, 3)])
def test_append(awq, T, hq, hkv, d, rot, page, layout):
    q, k, v = fused(T, hq, hkv, d, "bf16", T + d)
    pages = 2 * T // page + 3
    g = torch.Generator().manual_seed(1)
    if layout == "page, token, head":
        kc, vc = (torch.randn((pages, page, hkv, d), generator=g).bfloat16().cuda() for _ in range(2))
    elif layout == "page, head, token":
        kc, vc = (torch.randn((pages, hkv, page, d), generator=g).bfloat16().cuda().transpose(1, 2) for _ in range(2))
    else:
        both = torch.randn((pages, 2, page, hkv, d), generator=g).bfloat16().cuda()
        kc, vc = both[:, 0], both[:, 1]
    k0, v0 = f64(kc), f64(vc)
    rng = np.random.default_rng(T)
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    if T > 3:
        slots[1], slots[2] = -1, pages * page  # kept nowhere
    pos = rng.integers(0, 700, T).astype(np.int32)
    table = awq.awq_rope_table(700, rot)
    qo = awq.awq_rope_append(q, k, v, torch.from_numpy(pos).cuda(), table, kc, vc, torch.from_numpy(slots).cuda())
    wq, wk = awq.awq_rope(q, k, torch.from_numpy(pos).cuda(), table)
    assert torch.equal(qo, wq)
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            k0[s // page, s % page], v0[s // page, s % page] = f64(wk[t]), f64(v[t])
    assert np.array_equal(f64(kc), k0) and np.array_equal(f64(vc), v0)


def test_append_offsets_past_32_bits(awq):
    # the last page of a cache of over 2^32 elements
    d, page = 256, 64
    pages = (1 << 32) // (page * d) + 2
    kc, vc = (torch.empty((pages, page, 1, d), dtype=torch.float16, device="cuda") for _ in range(2))
    q, k, v = fused(2, 1, 1, d, "fp16", 9)
    pos = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    table = awq.awq_rope_table(8, d)
    last = pages * page - 1
    awq.awq_rope_append(q, k, v, pos, table, kc, vc, torch.tensor([last, 0], dtype=torch.int32, device="cuda"))
    assert torch.equal(kc[-1, -1], awq.awq_rope(q, k, pos, table)[1][0]) and torch.equal(vc[-1, -1], v[0])
    assert torch.equal(vc[0, 0], v[1])


def test_refusals(awq):
    q, k, v = fused(4, 2, 1, 64, "fp16", 1)
    table, pos = awq.awq_rope_table(16, 64), torch.zeros((4,), dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        awq.awq_rope(q.float(), k, pos, table)
    with pytest.raises(TypeError):
        awq.awq_rope(q, k.bfloat16(), pos, table)
    with pytest.raises(TypeError):
        awq.awq_rope(q, k, pos.long(), table)
    with pytest.raises(ValueError):
        awq.awq_rope(q, k, pos[:3], table)
    with pytest.raises(ValueError):
        awq.awq_rope(q.transpose(1, 2), k, pos, table)
    with pytest.raises(ValueError):
        awq.awq_rope(q, k, pos.cpu(), table)
    with pytest.raises(awq.AwqError):
        awq.awq_rope(q, k, pos, awq.awq_rope_table(16, 128))  # more than the head holds
    with pytest.raises(ValueError):
        awq.awq_rope_table(16, 64, scaling="other")
    with pytest.raises(ValueError):  # neither in place nor apart from its input
        awq.awq_rope(q, k, pos, table, q_out=q.as_strided((4, 2, 64), (128, 64, 1)))
    cache = torch.empty((2, 4, 1, 64), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        awq.awq_rope_append(q, k, v, pos, table, cache, cache.transpose(0, 1).contiguous().transpose(0, 1), pos)
    with pytest.raises(ValueError):
        awq.awq_rope_append(q, k, v, pos, table, cache.expand(2, 4, 3, 64), cache.expand(2, 4, 3, 64), pos)


def test_empty(awq):
    q, k, _ = fused(0, 2, 1, 64, "fp16", 1)
    qo, ko = awq.awq_rope(q, k, torch.zeros((0,), dtype=torch.int32, device="cuda"), awq.awq_rope_table(16, 64))
    assert qo.shape == (0, 2, 64) and ko.shape == (0, 1, 64)
