"""Host-only refusals of the operators between a layer's linears: bad arguments are found before any
device access.  The addresses are fake; no call here reaches a launch."""
import ctypes

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


def test_rope_table(lib):
    def call(n=16, rot=8, base=1e4, scaling=0, factor=1.0, original=0, p0=1.0, p1=1.0, af=1.0, table=A):
        return lib.awq_rope_table(table, n, rot, base, scaling, factor, original, p0, p1, af, None)
    assert call() == DEVICE and call(n=0, table=None) == 0
    assert call(rot=7) == INVALID and call(rot=0) == INVALID and call(n=-1) == INVALID
    assert call(base=1.0) == INVALID and call(base=float("nan")) == INVALID and call(af=0.0) == INVALID
    assert call(scaling=5) == INVALID and call(scaling=1, factor=0.0) == INVALID
    assert call(scaling=2, rot=2, factor=2.0) == INVALID
    assert call(scaling=3, factor=2.0) == INVALID                              # no original_max_position
    assert call(scaling=3, factor=2.0, original=64, p0=1.0, p1=32.0) == INVALID
    assert call(scaling=4, factor=2.0, original=64, p0=4.0, p1=1.0) == INVALID
    assert call(scaling=4, factor=2.0, original=64, p0=1.0, p1=4.0) == DEVICE
    assert call(table=None) == INVALID and call(table=ODD) == MISALIGNED and call(n=1 << 31) == SHAPE


def cache(**kw):
    from w4a16_weight_only_gb300._binding import PagedKV
    d = dict(k=0x100000, v=0x200000, num_pages=4, page_size=16, heads=2, head_dim=64, page_stride=16 * 128, token_stride=128,
             head_stride=64)
    d.update(kw)
    return PagedKV(*(d[n] for n, _ in PagedKV._fields_))


def rope(lib, T=4, Hq=4, Hkv=2, D=64, rot=64, mp=32, q=A, k=A, pos=A, table=A, qo=B, ko=B, dtype=0):
    return lib.awq_rope(q, k, pos, table, T, Hq, Hkv, D, rot, mp, Hq * D, D, Hkv * D, D, qo, ko, 0, dtype, None)


def append(lib, T=4, Hkv=2, D=64, kv=None, v=A, slots=A, c=True):
    kv = kv or cache()
    return lib.awq_rope_append(A, A, v, A, A, T, 4, Hkv, D, D, 32, 4 * D, D, Hkv * D, D, Hkv * D, D, B,
                               ctypes.byref(kv) if c else None, slots, 0, 0, None)


def test_rope(lib):
    assert rope(lib) == DEVICE and rope(lib, T=0, q=None, k=None, pos=None, table=None, qo=None, ko=None) == 0
    assert rope(lib, rot=65) == INVALID and rope(lib, rot=66) == INVALID and rope(lib, rot=0) == INVALID
    assert rope(lib, T=-1) == INVALID and rope(lib, dtype=1) == INVALID and rope(lib, dtype=9) == INVALID
    assert rope(lib, q=None) == INVALID and rope(lib, ko=None) == INVALID and rope(lib, table=None) == INVALID
    assert rope(lib, q=P(0x100001)) == MISALIGNED and rope(lib, pos=ODD) == MISALIGNED
    assert rope(lib, T=1 << 31) == SHAPE and rope(lib, Hq=1 << 17) == SHAPE
    assert append(lib) == DEVICE and append(lib, c=False) == INVALID and append(lib, Hkv=1) == INVALID
    assert append(lib, v=None) == INVALID and append(lib, slots=None) == INVALID
    assert append(lib, kv=cache(page_size=0)) == INVALID and append(lib, kv=cache(k=None)) == INVALID
    assert append(lib, kv=cache(token_stride=-128)) == INVALID and append(lib, kv=cache(num_pages=1 << 30)) == SHAPE


def attention(lib, B_=2, n=1, Hq=4, kv=None, prefix=20, W=2, max_len=32, q=A, out=B, pp=A, pages=A, lens=A, ws=A, wsb=1 << 30,
              stride=64, dtype=0):
    kv = kv or cache()
    return lib.awq_attention_shared(q, B_, n, Hq, Hq * stride, Hq * stride, stride, ctypes.byref(kv), pp, prefix, pages, W, W,
                                    lens, max_len, 0.125, out, dtype, ws, wsb, None)


def test_attention(lib):
    assert attention(lib) == DEVICE and attention(lib, B_=0, q=None, out=None) == 0
    assert attention(lib, Hq=3) == INVALID and attention(lib, prefix=-1) == INVALID and attention(lib, max_len=33) == INVALID
    assert attention(lib, kv=cache(head_dim=80)) == SHAPE and attention(lib, prefix=1 << 31) == SHAPE
    assert attention(lib, prefix=(1 << 31) - 255) == SHAPE
    assert attention(lib, q=None) == INVALID and attention(lib, pp=None) == INVALID and attention(lib, lens=None) == INVALID
    assert attention(lib, prefix=0, pp=None) == DEVICE
    assert attention(lib, max_len=0, pages=None, lens=None) == DEVICE
    assert attention(lib, q=ODD) == MISALIGNED and attention(lib, stride=65) == MISALIGNED
    assert attention(lib, kv=cache(token_stride=130)) == MISALIGNED and attention(lib, kv=cache(k=0x100008)) == MISALIGNED
    assert attention(lib, dtype=1) == INVALID
    n = ctypes.c_size_t(0)
    size = lib.awq_attention_shared_workspace_size
    assert size(2, 1, 4, 2, 64, 20, 32, ctypes.byref(n)) == 0 and n.value >= 2 * 4 * 2 * (64 + 2) * 4
    assert size(0, 1, 4, 2, 64, 20, 32, ctypes.byref(n)) == 0 and n.value == 0
    assert size(2, 1, 4, 2, 64, 20, 32, None) == INVALID and size(2, 1, 5, 2, 64, 20, 32, ctypes.byref(n)) == INVALID


def route(lib, T=4, E=8, k=2, dtype=0, groups=1, tg=1, gb=1, logits=A, bias=None, w=B, e=B):
    return lib.awq_moe_route(logits, T, E, E, dtype, k, 0, bias, groups, tg, gb, 1, 1.0, w, e, None)


def test_route(lib):
    assert route(lib) == DEVICE and route(lib, T=0, logits=None, w=None, e=None) == 0
    assert route(lib, E=0) == INVALID and route(lib, E=1025) == INVALID and route(lib, k=0) == INVALID
    assert route(lib, k=9) == INVALID and route(lib, E=64, k=33) == INVALID and route(lib, groups=3) == INVALID
    assert route(lib, groups=4, tg=1, k=3) == INVALID and route(lib, groups=2, tg=3) == INVALID
    assert route(lib, groups=2, tg=1, gb=3) == INVALID and route(lib, dtype=3) == INVALID
    assert route(lib, logits=None) == INVALID and route(lib, w=ODD) == MISALIGNED and route(lib, dtype=1, logits=ODD) == MISALIGNED
    assert route(lib, bias=ODD) == MISALIGNED


def test_dispatch_and_combine(lib):
    def dispatch(T=4, W=64, k=2, E=8, x=A, ids=A, routed=B, offsets=B, rows=B, ws=A, wsb=1 << 20):
        return lib.awq_moe_dispatch(x, T, W, W, ids, k, E, routed, offsets, rows, ws, wsb, None)
    assert dispatch() == DEVICE and dispatch(T=-1) == INVALID and dispatch(E=0) == INVALID and dispatch(E=4097) == INVALID
    assert dispatch(k=0) == INVALID and dispatch(k=1025) == INVALID and dispatch(x=None) == INVALID
    assert dispatch(W=0, x=None, routed=None) == DEVICE and dispatch(offsets=None) == INVALID
    assert dispatch(ids=ODD) == MISALIGNED and dispatch(T=1 << 30, k=4) == SHAPE
    n = ctypes.c_size_t(0)
    assert lib.awq_moe_dispatch_workspace_size(4, 2, 8, ctypes.byref(n)) == 0 and n.value >= 4 * 2 * 4
    assert lib.awq_moe_dispatch_workspace_size(4, 2, 8, None) == INVALID

    def combine(R=8, W=64, T=4, k=2, y=A, w=A, rows=A, base=None, out=B, dtype=0):
        return lib.awq_moe_combine(y, R, W, w, rows, T, k, base, out, dtype, None)
    assert combine() == DEVICE and combine(T=0, y=None, w=None, rows=None, out=None) == 0 and combine(W=0) == 0
    assert combine(k=0, w=None, rows=None) == DEVICE and combine(R=0, y=None) == DEVICE
    assert combine(R=-1) == INVALID and combine(k=1025) == INVALID and combine(y=None) == INVALID and combine(out=None) == INVALID
    assert combine(dtype=1) == INVALID and combine(rows=ODD) == MISALIGNED and combine(y=P(0x100001)) == MISALIGNED
    assert combine(R=1 << 31) == SHAPE


def test_strides_of_single_entries_do_not_matter(lib):
    # a dimension of one entry is never stepped along, whatever its stride
    def call(B=2, n=2, Hq=4, strides=(512, 256, 64), **kv):
        c = cache(**kv)
        return lib.awq_attention_shared(A, B, n, Hq, *strides, ctypes.byref(c), A, 10, A, 2, 2, A, 2, 0.125, P(0x200000), 0, A, 1 << 30,
                                        None)
    assert call() == DEVICE
    assert call(strides=(513, 256, 64)) == MISALIGNED and call(B=1, strides=(513, 256, 64)) == DEVICE
    assert call(strides=(512, 257, 64)) == MISALIGNED and call(n=1, strides=(512, 257, 64)) == DEVICE
    assert call(Hq=2, heads=1, strides=(512, 256, 65)) == MISALIGNED and call(Hq=1, heads=1, strides=(512, 256, 65)) == DEVICE
    assert call(head_stride=65) == MISALIGNED and call(heads=1, head_stride=65) == DEVICE
    assert call(token_stride=129) == MISALIGNED and call(page_size=1, token_stride=129) == DEVICE
    assert call(page_stride=2049) == MISALIGNED and call(num_pages=1, page_stride=2049) == DEVICE
    assert call(heads=1, head_stride=-1) == DEVICE and call(head_stride=-64) == INVALID
