"""GPU parity of the 4-bit cache's append, read and attention against the oracle.

Append and read: every operation is defined to the bit (fp32, each rounded by itself), so the cache's bytes
and the rotated queries are compared for equality.

Attention, per element: the result's rounding u |y| (u = 2^-11 fp16, 2^-8 bf16; fp16 results below the normal
range round to a multiple of 2^-24); the rounding of a value's factor, probability times scale, to fp16's 11
bits: 2^-11 relative, and for factors below its normal range 2^-25 of a factor whose unit is the largest
scale (twice, as a power of two) over the sum of probabilities, at least 2^7 (a maximum's probability is kept
as 2^7 or more): N * 15 * 2 * 2^-32 of the largest scale; fp32 arithmetic: a logit is a sum of D products
(2^-22 (D + 8) Z, Z the largest scale * sum |q| (code * s + |m|); it moves p by that relative amount, twice
through the denominator), sums over N keys (2^-22 (N + 64) relative).  All but the first are relative to
sum_j p_j (code * s + |m|)."""
import math

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


def f32(t):
    return t.detach().cpu().float().numpy()


def f64(t):
    return t.detach().cpu().double().numpy()


def equal(got, want):
    """Bit equality of fp32 values, NaN equal to NaN."""
    return np.array_equal(got, want, equal_nan=True)


# ------------------------------------------------------------------------- append and read ----

# T, hq, hkv, D, group, rot, interleaved, page
APPEND = [
    (1, 1, 1, 64, 64, 64, False, 16),
    (5, 8, 2, 128, 128, 128, False, 16),
    (7, 6, 2, 96, 32, 96, True, 32),
    (33, 4, 4, 128, 32, 64, True, 48),
    (19, 14, 2, 256, 64, 256, False, 16),
    (6, 2, 1, 256, 128, 128, True, 64),
    (40, 3, 3, 64, 32, 30, False, 16),      # pairs that do not fall on vectors
    (9, 5, 1, 128, 64, 2, False, 32),
    (3, 2, 2, 96, 32, 50, False, 16),
]


def rows(T, hq, hkv, D, dtype, seed, size=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    width = (hq + 2 * hkv) * D
    qkv = (size * torch.randn((T, width + pad), generator=g)).to(DT[dtype]).cuda()
    return (qkv[:, :hq * D].view(T, hq, D) if not pad else qkv[:, :hq * D].unflatten(1, (hq, D)),
            qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D)), qkv[:, (hq + hkv) * D:width].unflatten(1, (hkv, D)))


def expected(k, v, positions, table, group, dtype, interleaved):
    kf = f32(k) if table is None else step.rotate(f32(k), positions, f32(table), dtype, interleaved)
    return step.quantize(kf, group, dtype), step.quantize(f32(v), group, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_and_read(awq, case, dtype):
    T, hq, hkv, D, group, rot, interleaved, page = APPEND[case]
    q, k, v = rows(T, hq, hkv, D, dtype, case, pad=0 if case % 2 else 8)
    table = awq.awq_rope_table(256, rot)
    rng = np.random.default_rng(case)
    positions = rng.integers(0, 256, T)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T]
    if T > 4:
        slots[T // 2] = -1
    before = torch.from_numpy(rng.integers(0, 256, (pages, hkv, awq.awq_kv4_page_bytes(page, D, group)), dtype=np.uint8))
    cache = before.cuda()
    out = awq.awq_rope_append_kv4(q, k, v, torch.from_numpy(positions).int().cuda(), table, cache,
                                  torch.from_numpy(slots).int().cuda(), group_size=group, interleaved=interleaved)
    assert equal(f32(out), step.rotate(f32(q), positions, f32(table), dtype, interleaved))
    kq, vq = expected(k, v, positions, table, group, dtype, interleaved)
    want = before.numpy().copy()
    for t in range(T):
        step.store(want, page, int(slots[t]), [x[t] for x in kq], [x[t] for x in vq], dtype)
    assert np.array_equal(cache.cpu().numpy(), want)
    rk, rv = awq.awq_kv4_read(cache, torch.from_numpy(slots).int().cuda(), D, group_size=group, dtype=DT[dtype])
    for got, quant in ((rk, kq), (rv, vq)):
        code, scale, low = quant
        value = step.round_to((code.reshape(*scale.shape, -1).astype(np.float32) * scale[..., None]).astype(np.float32) + low[..., None],
                              dtype).reshape(code.shape)
        value[slots < 0] = 0
        assert equal(f32(got), value)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_extremes(awq, dtype):
    # constant groups, the largest and smallest numbers, infinities and NaN: their group alone reads NaN
    T, H, D, group = 6, 2, 128, 32
    top = 65504.0 if dtype == "fp16" else 3.3895313892515355e38
    k = torch.randn((T, H, D), generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    v = k.flip(0).clone()
    k[0] = 1.5
    k[1, :, ::2], k[1, :, 1::2] = top, -top
    k[2] *= 2.0 ** -22 if dtype == "fp16" else 2.0 ** -130
    k[3, 0, 40], k[3, 1, 0], k[3, 1, 127] = float("inf"), float("nan"), -float("inf")
    v[4] = 0.0
    k, v = k.cuda(), v.cuda()
    cache = torch.zeros((1, H, awq.awq_kv4_page_bytes(16, D, group)), dtype=torch.uint8, device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    assert awq.awq_rope_append_kv4(None, k, v, None, None, cache, slots, group_size=group) is None
    rk, rv = awq.awq_kv4_read(cache, slots, D, group_size=group, dtype=DT[dtype])
    for got, x in ((rk, k), (rv, v)):
        code, scale, low = step.quantize(f32(x), group, dtype)
        with np.errstate(all="ignore"):
            value = step.round_to((code.reshape(*scale.shape, -1).astype(np.float32) * scale[..., None]) + low[..., None], dtype)
        assert equal(f32(got), value.reshape(code.shape))
    assert np.isnan(f32(rk)[3, 0, 32:64]).all() and np.isfinite(f32(rk)[3, 0, :32]).all()
    assert (f32(rk)[0] == 1.5).all() and (f32(rv)[4] == 0).all()


def test_append_outside_the_table_or_the_cache(awq):
    q, k, v = rows(3, 2, 1, 64, "fp16", 3)
    table = awq.awq_rope_table(16, 32)
    cache = torch.full((2, 1, awq.awq_kv4_page_bytes(16, 64, 32)), 7, dtype=torch.uint8, device="cuda")
    slots = torch.tensor([32, -5, 31], dtype=torch.int32, device="cuda")
    before = cache.clone()
    out = awq.awq_rope_append_kv4(q, k, v, torch.tensor([0, 1, 16], dtype=torch.int32, device="cuda"), table, cache, slots,
                                  group_size=32)
    assert torch.isnan(out[2, :, :32]).all() and torch.equal(out[2, :, 32:], q[2, :, 32:])
    rk, rv = awq.awq_kv4_read(cache, slots, 64, group_size=32)
    assert torch.isnan(rk[2, :, :32]).all() and torch.isfinite(rk[2, :, 32:]).all() and (rk[:2] == 0).all() and (rv[:2] == 0).all()
    assert torch.equal(cache[0], before[0])


def test_append_in_place_and_strided_cache(awq):
    # q rotated in place; a cache whose layers lie between its pages and whose heads are apart
    T, hq, hkv, D = 20, 4, 2, 128
    q, k, v = rows(T, hq, hkv, D, "bf16", 9)
    table, nbytes = awq.awq_rope_table(64, D), awq.awq_kv4_page_bytes(16, D)
    store = torch.zeros((3, 2, 3, nbytes + 32), dtype=torch.uint8, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    dense = torch.zeros((3, hkv, nbytes), dtype=torch.uint8, device="cuda")
    want = awq.awq_rope_append_kv4(q, k, v, pos, table, dense, pos)
    view = store[:, 1, :hkv, :nbytes]
    got = awq.awq_rope_append_kv4(q, k, v, pos, table, view, pos, q_out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(q, want) and torch.equal(view, dense)
    assert (store[:, 0] == 0).all() and (store[:, 1, hkv:] == 0).all() and (store[..., nbytes:] == 0).all()
    for a, b in zip(awq.awq_kv4_read(view, pos, D, dtype=torch.bfloat16), awq.awq_kv4_read(dense, pos, D, dtype=torch.bfloat16)):
        assert torch.equal(a, b)


# ----------------------------------------------------------------------------- attention ----

def make(awq, B, n, hq, hkv, D, group, lens, page, dtype, seed=0, sharp=1.0, spare=0, shift=0.0):
    """A cache whose cells hold 0xff (NaN scales and minima) wherever no token was written."""
    rng = np.random.default_rng(seed)
    per = max(1, -(-max(list(lens) + [1]) // page)) + spare
    total = B * per + 2
    pages = rng.permutation(total)[:B * per].reshape(B, per).astype(np.int32)
    cache = torch.full((total, hkv, awq.awq_kv4_page_bytes(page, D, group)), 255, dtype=torch.uint8, device="cuda")
    keys, values = [], []
    for b in range(B):
        pair = []
        for which in range(2):
            x = rng.standard_normal((lens[b], hkv, D))
            if which == 0:
                x = x + shift * rng.standard_normal((1, hkv, D))
            pair.append(torch.from_numpy(x).to(DT[dtype]).cuda())
        at = np.arange(lens[b])
        slots = pages[b, at // page] * page + at % page
        if lens[b]:
            awq.awq_rope_append_kv4(None, *pair, None, None, cache, torch.from_numpy(slots.astype(np.int32)).cuda(), group_size=group)
        for x, to in zip(pair, (keys, values)):
            code, scale, low = step.quantize(f32(x), group, dtype)
            to.append((step.dequantize(code, scale, low), step.dequantize(code, scale, np.abs(low)), scale))
    q = torch.from_numpy(sharp * rng.standard_normal((B, n, hq, D))).to(DT[dtype]).cuda()
    call = dict(q=q, cache=cache, pages=torch.from_numpy(pages).cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                group_size=group)
    return call, keys, values


def check(out, call, keys, values, dtype, scale=None, window=0, sinks=0):
    q = f64(call["q"]) if call["q"].dim() == 4 else f64(call["q"])[:, None]
    D, lens = q.shape[-1], call["lens"].tolist()
    scale = 1 / math.sqrt(D) if scale is None else scale
    want, spread, z = step.attention(q, keys, values, lens, scale, window, sinks)
    N = max(lens + [0])
    largest = max([float(v[2].max()) for v in values if v[2].size] + [0.0])
    fp32 = 2 * 2.0 ** -22 * (D + 8) * z + 2.0 ** -22 * (N + 64)
    tol = U[dtype] * np.abs(want) + (2.0 ** -11 + fp32) * spread * (1 + U[dtype]) + N * 30 * 2.0 ** -32 * largest
    tol = tol + (2.0 ** -24 if dtype == "fp16" else 0)
    got = f64(out).reshape(want.shape)
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())


# B, n, hq, hkv, D, group, lens, page, window, sinks
CASES = [
    (1, 1, 1, 1, 64, 64, [1], 16, 0, 0),                    # one key
    (2, 1, 8, 2, 128, 128, [0, 0], 16, 0, 0),               # nothing seen: zeros
    (3, 1, 8, 1, 128, 64, [5, 0, 200], 16, 0, 0),           # a slot without a sequence
    (2, 1, 4, 4, 96, 32, [17, 64], 48, 0, 0),
    (4, 1, 16, 2, 64, 32, [1, 15, 16, 33], 16, 0, 0),       # around a tile
    (2, 3, 6, 2, 96, 32, [3, 50], 16, 0, 0),                # several new tokens, causal
    (2, 5, 14, 2, 128, 32, [4, 131], 16, 0, 0),             # a sequence shorter than its new tokens: a row sees nothing
    (1, 1, 64, 1, 128, 128, [90], 64, 0, 0),                # one key/value head for all
    (2, 2, 40, 1, 64, 64, [2, 34], 32, 0, 0),               # 80 rows of a head
    (2, 1, 8, 2, 256, 64, [31, 70], 16, 0, 0),
    (1, 20, 4, 4, 256, 128, [40], 16, 0, 0),
    (2, 1, 4, 2, 256, 32, [9, 100], 16, 0, 0),
    (1, 1, 2, 1, 128, 128, [6000], 16, 0, 0),               # cut along the keys, few heads
    (33, 1, 8, 2, 128, 128, [(37 * i) % 241 for i in range(33)], 16, 0, 0),
    (9, 1, 4, 4, 64, 64, [700 + 31 * i for i in range(9)], 64, 0, 0),
    (40, 1, 16, 8, 64, 32, [(53 * i) % 300 for i in range(40)], 16, 0, 0),   # more units than blocks at a time
    (3, 1, 8, 2, 128, 64, [2500, 40, 3000], 16, 0, 0),      # tables too long for a unit per block
    (2, 5, 8, 2, 96, 32, [3000, 2200], 16, 0, 0),
    (2, 1, 8, 2, 128, 128, [300, 77], 16, 64, 0),           # windows
    (2, 1, 8, 2, 128, 64, [300, 77], 16, 50, 4),
    (3, 1, 8, 8, 64, 32, [1000, 5, 130], 32, 100, 20),      # first tokens beyond a tile
    (2, 4, 8, 2, 128, 128, [500, 6], 16, 1, 1),             # a window of the token itself
    (2, 4, 6, 1, 96, 32, [333, 40], 16, 37, 3),
    (2, 1, 4, 1, 128, 128, [200, 100], 16, 150, 60),        # window and first tokens meet in one of the two
    (2, 2, 4, 1, 256, 64, [200, 100], 16, 1000, 2000),      # both longer than the sequence
    (1, 70, 4, 2, 128, 128, [70], 16, 0, 0),                # a prompt
    (1, 130, 2, 1, 64, 64, [200], 16, 24, 2),               # a prompt under a window
    (2, 3, 8, 2, 128, 128, [5000, 2100], 16, 2300, 70),     # a long window, cut along the keys
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(awq, case, dtype):
    B, n, hq, hkv, D, group, lens, page, window, sinks = CASES[case]
    call, keys, values = make(awq, B, n, hq, hkv, D, group, lens, page, dtype, seed=case, shift=1.0 if case % 2 else 0.0)
    out = awq.awq_attention_kv4(**call, window=window, sinks=sinks)
    check(out, call, keys, values, dtype, window=window, sinks=sinks)
    assert torch.equal(out, awq.awq_attention_kv4(**call, window=window, sinks=sinks))


def test_many_short_sequences(awq):
    # more sequences than entries of a block's table of lengths, several of them in a warp's share, some empty
    B = 700
    lens = [(7 * i) % 37 for i in range(B)]
    call, keys, values = make(awq, B, 1, 8, 4, 64, 64, lens, 16, "fp16", seed=18)
    out = awq.awq_attention_kv4(**call)
    some = list(range(0, B, 29)) + [B - 1]
    part = dict(call, q=call["q"][some], lens=call["lens"][some])
    check(out[some], part, [keys[i] for i in some], [values[i] for i in some], "fp16")
    assert (out[call["lens"] == 0] == 0).all() and torch.equal(out, awq.awq_attention_kv4(**call))


def test_pages_beyond_four_gigabytes(awq):
    # byte offsets of pages and cells pass 32 bits
    call, keys, values = make(awq, 2, 2, 8, 2, 128, 128, [90, 140], 64, "bf16", seed=17)
    nbytes = awq.awq_kv4_page_bytes(64, 128)
    far = (9 << 29) // (2 * nbytes)  # pages: 4.5 GiB in front
    cache = torch.empty((far + call["cache"].shape[0], 2, nbytes), dtype=torch.uint8, device="cuda")
    cache[far:] = call["cache"]
    check(awq.awq_attention_kv4(**dict(call, cache=cache, pages=call["pages"] + far)), call, keys, values, "bf16")
    slots = (call["pages"][1, :2].repeat_interleave(64) * 64 + torch.arange(128, device="cuda") % 64).int()
    k, v = awq.awq_kv4_read(call["cache"], slots, 128, dtype=torch.bfloat16)
    for got, want in zip(awq.awq_kv4_read(cache, slots + far * 64, 128, dtype=torch.bfloat16), (k, v)):
        assert torch.equal(got, want)
    awq.awq_rope_append_kv4(None, v, k, None, None, cache, slots + far * 64)
    awq.awq_rope_append_kv4(None, v, k, None, None, call["cache"], slots)
    assert torch.equal(cache[far:], call["cache"])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("sharp,scale", [(8.0, None), (1.0, 0.0), (1.0, -0.2), (30.0, 0.5)])
def test_logits(awq, dtype, sharp, scale):
    call, keys, values = make(awq, 2, 1, 8, 2, 128, 64, [150, 700], 16, dtype, seed=7, sharp=sharp)
    check(awq.awq_attention_kv4(**call, scale=scale), call, keys, values, dtype, scale=scale)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_values_of_very_different_sizes(awq, dtype):
    # tokens whose values are a thousand times larger come late, in the middle, or not at all
    call, keys, _ = make(awq, 3, 1, 4, 1, 128, 64, [300, 300, 300], 16, dtype, seed=11)
    rng = np.random.default_rng(12)
    values = []
    for b in range(3):
        x = rng.standard_normal((300, 1, 128)) * 2.0 ** -10
        if b < 2:
            x[290 if b == 0 else 150] *= 2.0 ** 14
        x = torch.from_numpy(x).to(DT[dtype]).cuda()
        at = np.arange(300)
        slots = torch.from_numpy((call["pages"].cpu().numpy()[b, at // 16] * 16 + at % 16).astype(np.int32)).cuda()
        k, _ = awq.awq_kv4_read(call["cache"], slots, 128, group_size=64, dtype=DT[dtype])
        awq.awq_rope_append_kv4(None, k, x, None, None, call["cache"], slots, group_size=64)
        for quant, to in ((f32(k), None), (f32(x), values)):
            code, scale, low = step.quantize(quant, 64, dtype)
            entry = (step.dequantize(code, scale, low), step.dequantize(code, scale, np.abs(low)), scale)
            if to is None:
                keys[b] = entry
            else:
                to.append(entry)
    check(awq.awq_attention_kv4(**call), call, keys, values, dtype)


def test_queries_of_any_size_bf16(awq):
    for sharp in (2.0 ** 60, 2.0 ** -60):
        call, keys, values = make(awq, 2, 1, 4, 2, 64, 32, [40, 90], 16, "bf16", seed=5, sharp=sharp)
        check(awq.awq_attention_kv4(**call, scale=0.125 / sharp), call, keys, values, "bf16", scale=0.125 / sharp)


def test_strided_queries_and_given_tensors(awq):
    call, keys, values = make(awq, 3, 2, 8, 2, 128, 128, [50, 3, 129], 16, "fp16", seed=2)
    wide = torch.zeros((3, 2, 12, 136), dtype=torch.float16, device="cuda")
    wide[:, :, 2:10, :128] = call["q"]
    table = torch.full((3, 20), 1 << 30, dtype=torch.int32, device="cuda")
    table[:, 3:3 + call["pages"].shape[1]] = call["pages"]
    call.update(q=wide[:, :, 2:10, :128], pages=table[:, 3:])  # entries past a sequence's pages are never looked up
    out = torch.empty((3, 2, 8, 128), dtype=torch.float16, device="cuda")
    ws = torch.full((awq.awq_attention_kv4_workspace_size(3, 2, 8, 2, 128) or 1,), 255, dtype=torch.uint8, device="cuda")
    got = awq.awq_attention_kv4(**call, out=out, workspace=ws)
    assert got.data_ptr() == out.data_ptr()
    check(out, call, keys, values, "fp16")
    call3 = dict(call, q=call["q"][:, 1])
    one = awq.awq_attention_kv4(**call3)
    check(one, call3, keys, values, "fp16")


def test_pages_behind_a_window_are_not_read(awq):
    call, keys, values = make(awq, 1, 1, 4, 1, 128, 128, [500], 16, "bf16", seed=4)
    call["pages"][0, 1:27] = -1  # tokens 16 .. 431
    check(awq.awq_attention_kv4(**call, window=60, sinks=5), call, keys, values, "bf16", window=60, sinks=5)


def test_bad_pages_and_lengths_stay_inside(awq):
    call, keys, values = make(awq, 3, 1, 8, 2, 128, 128, [100, 200, 60], 16, "fp16", seed=6)
    good = awq.awq_attention_kv4(**call)
    bad = dict(call, pages=call["pages"].clone(), lens=call["lens"].clone())
    bad["pages"][1, 3], bad["pages"][1, 4] = -7, 1 << 30
    out = awq.awq_attention_kv4(**bad)
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    bad["lens"][1] = 2 ** 31 - 1  # cut to what the pages hold
    bad["lens"][2] = -3
    out = awq.awq_attention_kv4(**bad)
    assert (out[2] == 0).all()  # the others' lengths move where a sequence's keys are cut: equal to rounding
    first = dict(call, q=call["q"][:1], lens=call["lens"][:1])
    check(out[:1], first, keys[:1], values[:1], "fp16")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rows_are_apart(awq, dtype):
    # a NaN key or value of a newer token stays with the rows that see it
    call, keys, values = make(awq, 2, 4, 8, 2, 128, 64, [60, 45], 16, dtype, seed=8)
    good = awq.awq_attention_kv4(**call)
    for where in ("k", "v"):
        b, j = 0, 58  # seen by the last two of the four
        page = int(call["pages"][b, j // 16])
        cache = call["cache"].clone()
        slot = torch.tensor([page * 16 + j % 16], dtype=torch.int32, device="cuda")
        k, v = awq.awq_kv4_read(cache, slot, 128, group_size=64, dtype=DT[dtype])
        (k if where == "k" else v)[0, :, 70] = float("nan")
        awq.awq_rope_append_kv4(None, k, v, None, None, cache, slot, group_size=64)
        out = awq.awq_attention_kv4(**dict(call, cache=cache))
        assert torch.equal(out[0, :2], good[0, :2]) and torch.equal(out[1], good[1])
        assert torch.isnan(out[0, 2:, :, 64:]).all()
        assert where == "v" or torch.isnan(out[0, 2:]).all()


def test_all_logits_minus_infinity(awq):
    call, keys, values = make(awq, 1, 1, 2, 1, 64, 64, [20], 16, "fp16", seed=3)
    call["q"][0, 0, 0] = 60000.0
    k = torch.full((20, 1, 64), -60000.0, dtype=torch.float16, device="cuda")
    slots = call["pages"][0, :1].repeat(20) * 16
    slots = (call["pages"][0].repeat_interleave(16)[:20] * 16 + torch.arange(20, device="cuda") % 16).int()
    _, v = awq.awq_kv4_read(call["cache"], slots, 64, group_size=64)
    awq.awq_rope_append_kv4(None, k, v, None, None, call["cache"], slots, group_size=64)
    out = awq.awq_attention_kv4(**call, scale=1e36)
    assert torch.isnan(out[0, 0, 0]).all()


def test_waits_that_give_up(awq):
    # as if no copy arrived in time: an error status, and the next call is right
    call, keys, values = make(awq, 3, 1, 8, 2, 128, 128, [100, 900, 60], 16, "bf16", seed=13)
    awq.selftest_attention_give_up(True)
    try:
        awq.awq_attention_kv4(**call)
    finally:
        awq.selftest_attention_give_up(False)
    with pytest.raises(awq.AwqError):
        awq.device_status()
    check(awq.awq_attention_kv4(**call), call, keys, values, "bf16")


def test_empty(awq):
    cache = torch.zeros((1, 2, awq.awq_kv4_page_bytes(16, 64, 64)), dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.zeros((0, 4, 64), dtype=torch.float16, device="cuda")
    assert awq.awq_attention_kv4(q, cache, torch.zeros((0, 3), **i32), torch.zeros((0,), **i32), group_size=64).shape == (0, 4, 64)
    q = torch.ones((2, 4, 64), dtype=torch.float16, device="cuda")
    out = awq.awq_attention_kv4(q, cache, torch.zeros((2, 0), **i32), torch.tensor([0, 5], **i32), group_size=64)
    assert (out == 0).all()  # a table without pages: no keys
    none = torch.zeros((0,), **i32)
    assert awq.awq_kv4_read(cache, none, 64, group_size=64)[0].shape == (0, 2, 64)
    k = torch.zeros((0, 2, 64), dtype=torch.float16, device="cuda")
    assert awq.awq_rope_append_kv4(None, k, k, None, None, cache, none, group_size=64) is None


def test_graph_and_streams(awq):
    # captured and replayed with new contents, on a stream of its own, beside eager calls of another
    call, keys, values = make(awq, 4, 1, 8, 2, 128, 128, [900, 33, 500, 1], 16, "bf16", seed=21)
    want = awq.awq_attention_kv4(**call)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        awq.awq_attention_kv4(**call)
    torch.cuda.synchronize()
    ws = torch.empty((awq.awq_attention_kv4_workspace_size(4, 1, 8, 2, 128) or 1,), dtype=torch.uint8, device="cuda")
    graph, lens = torch.cuda.CUDAGraph(), call["lens"].clone()
    with torch.cuda.graph(graph):
        out = awq.awq_attention_kv4(**call, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    call["lens"].copy_(torch.tensor([10, 20, 0, 1], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    check(out, call, [(k[0][:n], k[1][:n], k[2][:n]) for k, n in zip(keys, [10, 20, 0, 1])],
          [(v[0][:n], v[1][:n], v[2][:n]) for v, n in zip(values, [10, 20, 0, 1])], "bf16")
    call["lens"].copy_(lens)
    with torch.cuda.stream(side):
        again = [awq.awq_attention_kv4(**call) for _ in range(3)]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.equal(a, want) for a in again)
