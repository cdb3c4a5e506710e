"""Host-only checks of the operators around a 4-bit cache: refusals found before any device access (the
addresses are fake; no call here reaches a launch), and the layout of a tile."""
import ctypes

import numpy as np
import pytest

INVALID, SHAPE, MISALIGNED, DEVICE = 1, 2, 3, 4
P = ctypes.c_void_p
A, B, ODD = P(0x100000), P(0x200000), P(0x100002)


@pytest.fixture(scope="module")
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("host-only checks with fake device addresses; a CUDA device is present")
    from w4a16_weight_only_gb300 import build
    build.build()
    from w4a16_weight_only_gb300 import _binding
    return _binding.load_library()


def cache(**kw):
    from w4a16_weight_only_gb300._binding import Kv4Cache
    d = dict(data=0x100000, num_pages=4, page_size=16, heads=2, head_dim=64, group_size=32, page_stride=2 * 16 * 80, head_stride=16 * 80)
    d.update(kw)
    return Kv4Cache(*(d[n] for n, _ in Kv4Cache._fields_))


BAD_CACHES = [(dict(data=None), INVALID), (dict(num_pages=-1), INVALID), (dict(page_size=0), INVALID), (dict(page_size=24), SHAPE),
              (dict(heads=0), INVALID), (dict(head_dim=80), SHAPE), (dict(group_size=0), INVALID), (dict(group_size=16), SHAPE),
              (dict(head_dim=96, group_size=64), SHAPE), (dict(head_dim=64, group_size=128), SHAPE),
              (dict(num_pages=1 << 28), SHAPE), (dict(page_stride=-16), INVALID), (dict(page_stride=8), MISALIGNED),
              (dict(head_stride=1288), MISALIGNED), (dict(data=0x100008), MISALIGNED)]


def test_page_bytes(lib):
    n = ctypes.c_size_t(0)
    assert lib.awq_kv4_page_bytes(64, 128, 64, ctypes.byref(n)) == 0 and n.value == 64 * (128 + 16)
    assert lib.awq_kv4_page_bytes(16, 96, 32, ctypes.byref(n)) == 0 and n.value == 16 * 120
    assert lib.awq_kv4_page_bytes(16, 128, 64, None) == INVALID and lib.awq_kv4_page_bytes(8, 128, 64, ctypes.byref(n)) == SHAPE
    assert lib.awq_kv4_page_bytes(16, 128, 48, ctypes.byref(n)) == SHAPE and lib.awq_kv4_page_bytes(-16, 128, 64, ctypes.byref(n)) == INVALID


def append(lib, T=4, Hq=4, Hkv=2, D=64, rot=64, mp=32, q=A, k=A, v=A, pos=A, table=A, qo=B, kv=None, slots=A, dtype=0, c=True):
    kv = kv or cache()
    return lib.awq_rope_append_kv4(q, k, v, pos, table, T, Hq, Hkv, D, rot, mp, Hq * D, D, Hkv * D, D, Hkv * D, D, qo,
                                   ctypes.byref(kv) if c else None, slots, 0, dtype, None)


def test_append(lib):
    assert append(lib) == DEVICE and append(lib, T=0, q=None, k=None, v=None, pos=None, slots=None, qo=None) == 0
    assert append(lib, table=None, pos=None, rot=0) == DEVICE and append(lib, Hq=0, q=None, qo=None) == DEVICE
    assert append(lib, rot=65) == INVALID and append(lib, rot=66) == INVALID and append(lib, rot=0) == INVALID
    assert append(lib, T=-1) == INVALID and append(lib, dtype=1) == INVALID and append(lib, c=False) == INVALID
    assert append(lib, Hkv=1) == INVALID and append(lib, D=128) == INVALID
    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(pos=None), dict(slots=None)):
        assert append(lib, **bad) == INVALID
    assert append(lib, q=P(0x100001)) == MISALIGNED and append(lib, pos=ODD) == MISALIGNED and append(lib, slots=ODD) == MISALIGNED
    assert append(lib, T=1 << 30) == SHAPE and append(lib, Hq=1 << 17) == SHAPE
    for kw, status in BAD_CACHES:
        assert append(lib, kv=cache(**kw), D=kw.get("head_dim", 64), rot=64) == status, kw
    # strides of single entries are not looked at
    assert append(lib, kv=cache(num_pages=1, page_stride=-3)) == DEVICE
    assert append(lib, Hkv=1, kv=cache(heads=1, head_stride=7)) == DEVICE


def test_read(lib):
    def read(T=4, slots=A, k=B, v=B, kv=None, dtype=0, c=True):
        kv = kv or cache()
        return lib.awq_kv4_read(ctypes.byref(kv) if c else None, slots, T, k, v, dtype, None)
    assert read() == DEVICE and read(T=0, slots=None, k=None, v=None) == 0 and read(c=False) == INVALID
    assert read(T=-1) == INVALID and read(slots=None) == INVALID and read(k=None) == INVALID and read(v=None) == INVALID
    assert read(dtype=1) == INVALID and read(T=1 << 30) == SHAPE and read(slots=ODD) == MISALIGNED and read(v=P(0x100001)) == MISALIGNED
    for kw, status in BAD_CACHES:
        assert read(kv=cache(**kw)) == status, kw


def attention(lib, B_=2, n=1, Hq=4, kv=None, W=2, q=A, out=B, pages=A, lens=A, window=0, sinks=0, ws=A, wsb=1 << 30, strides=None,
              dtype=0, c=True):
    kv = kv or cache()
    return lib.awq_attention_kv4(q, B_, n, Hq, *(strides or (n * Hq * 64, Hq * 64, 64)), ctypes.byref(kv) if c else None, pages, W, W,
                                 lens, window, sinks, 0.125, out, dtype, ws, wsb, None)


def test_attention(lib):
    assert attention(lib) == DEVICE and attention(lib, B_=0, q=None, out=None, lens=None) == 0 and attention(lib, c=False) == INVALID
    assert attention(lib, W=0, pages=None) == DEVICE and attention(lib, window=100, sinks=4) == DEVICE
    assert attention(lib, Hq=3) == INVALID and attention(lib, n=-1) == INVALID and attention(lib, W=-1) == INVALID
    assert attention(lib, W=1 << 28) == INVALID and attention(lib, window=-1) == INVALID and attention(lib, sinks=1 << 31) == INVALID
    assert attention(lib, q=None) == INVALID and attention(lib, out=None) == INVALID and attention(lib, pages=None) == INVALID
    assert attention(lib, lens=None) == INVALID and attention(lib, dtype=1) == INVALID
    assert attention(lib, q=ODD) == MISALIGNED and attention(lib, out=P(0x100008)) == MISALIGNED and attention(lib, lens=ODD) == MISALIGNED
    assert attention(lib, strides=(256, 256, 60)) == MISALIGNED and attention(lib, Hq=131072) == SHAPE
    assert attention(lib, B_=1, strides=(3, 256, 64)) == DEVICE and attention(lib, n=1, strides=(256, 3, 64)) == DEVICE
    for kw, status in BAD_CACHES:
        assert attention(lib, kv=cache(**kw)) == status, kw
    n = ctypes.c_size_t(0)
    size = lib.awq_attention_kv4_workspace_size
    assert size(2, 1, 4, 2, 64, ctypes.byref(n)) == 0 and size(0, 1, 4, 2, 64, ctypes.byref(n)) == 0 and n.value == 0
    assert size(2, 1, 4, 2, 64, None) == INVALID and size(2, 1, 5, 2, 64, ctypes.byref(n)) == INVALID
    assert size(2, 1, 4, 2, 80, ctypes.byref(n)) == SHAPE


def norm(lib, x=A, xs=64, r=A, rs=64, g=None, gs=0, pw=None, pb=None, w=A, b=None, T=4, W=64, kind=0, eps=1e-6, h=B, y=B, dtype=0):
    return lib.awq_residual_norm(x, xs, r, rs, g, gs, pw, pb, 1.0, w, b, T, W, kind, eps, h, y, dtype, None)


def test_norm(lib):
    assert norm(lib) == DEVICE and norm(lib, T=0, x=None, h=None, y=None) == 0 and norm(lib, W=0) == 0
    assert norm(lib, r=None) == DEVICE and norm(lib, w=None, y=None) == DEVICE and norm(lib, g=A, gs=64, pw=A, pb=A, b=A) == DEVICE
    assert norm(lib, x=None) == INVALID and norm(lib, h=None) == INVALID and norm(lib, y=None) == INVALID
    assert norm(lib, pb=A) == INVALID and norm(lib, w=None, b=A) == INVALID and norm(lib, kind=2) == INVALID
    assert norm(lib, eps=-1.0) == INVALID and norm(lib, eps=float("nan")) == INVALID and norm(lib, T=-1) == INVALID
    assert norm(lib, dtype=1) == INVALID and norm(lib, x=P(0x100001)) == MISALIGNED and norm(lib, T=1 << 31) == SHAPE
    assert norm(lib, h=A, rs=128) == INVALID and norm(lib, h=A, rs=64) == DEVICE  # in place needs dense rows
    assert norm(lib, y=A, xs=72) == INVALID and norm(lib, h=A, rs=128, T=1) == DEVICE


def moe(lib, T=4, H=256, k=2, E=4, I=128, G=128, x=A, ids=A, w=A, up=A, down=A, base=None, out=B, dtype=0, ws=A, wsb=1 << 24, zeros=A):
    return lib.awq_moe_layer(x, T, H, H, ids, w, k, E, I, G, up, zeros, A, down, zeros, A, base, out, dtype, ws, wsb, None)


def test_moe_layer(lib):
    assert moe(lib) == DEVICE and moe(lib, T=0, x=None, out=None) == 0 and moe(lib, H=0) == 0
    assert moe(lib, k=0, ids=None, w=None) == DEVICE and moe(lib, I=0, up=None) == DEVICE
    assert moe(lib, T=17) == INVALID and moe(lib, T=-1) == INVALID and moe(lib, k=33) == INVALID and moe(lib, E=0) == INVALID
    assert moe(lib, E=4097) == INVALID and moe(lib, G=0) == INVALID and moe(lib, G=-1) == INVALID
    assert moe(lib, H=100, G=4, I=8) == SHAPE and moe(lib, I=64) == SHAPE and moe(lib, H=192) == SHAPE
    assert moe(lib, x=None) == INVALID and moe(lib, ids=None) == INVALID and moe(lib, w=None) == INVALID and moe(lib, up=None) == INVALID
    assert moe(lib, out=A) == INVALID and moe(lib, dtype=1) == INVALID and moe(lib, zeros=None) == INVALID
    assert moe(lib, ids=ODD) == MISALIGNED and moe(lib, up=ODD) == MISALIGNED and moe(lib, base=P(0x100001)) == MISALIGNED
    assert moe(lib, H=1 << 20, I=1 << 20) == SHAPE
    n = ctypes.c_size_t(0)
    assert lib.awq_moe_layer_workspace_size(4, 2, 256, 128, ctypes.byref(n)) == 0 and n.value >= 4 * 2 * 128 * 2
    assert lib.awq_moe_layer_workspace_size(4, 2, 256, 128, None) == INVALID and lib.awq_moe_layer_workspace_size(17, 2, 256, 128, ctypes.byref(n)) == INVALID


@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (96, 32), (128, 32), (128, 128), (256, 64)])
def test_a_tile_holds_every_code_once(D, group):
    from oracle import step
    at = {(byte(D, r, e), e % 2) for byte in (step.key_byte, step.value_byte) for r in range(16) for e in range(D)}
    assert at == {(b, half) for b in range(16 * D) for half in range(2)}
    # the two elements of a byte are neighbours, and a token's writes share no byte with another's
    owner = {}
    for byte in (step.key_byte, step.value_byte):
        for r in range(16):
            for e in range(D):
                assert owner.setdefault((byte(D, r, e)), (r, e // 2)) == (r, e // 2)


def test_quantize_round_trip():
    from oracle import step
    rng = np.random.default_rng(0)
    x = step.round_to(rng.standard_normal((50, 128)), "fp16")
    code, scale, low = step.quantize(x, 32, "fp16")
    err = np.abs(step.dequantize(code, scale, low) - x).reshape(50, 4, 32)
    # half a step, and where the scale was rounded down the last step's rest
    assert (err <= 0.5 * scale[..., None] * (1 + 2.0 ** -20) + 15 * 2.0 ** -11 * scale[..., None]).all()
