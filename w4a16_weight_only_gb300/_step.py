"""Binding of the operators around a 4-bit key/value cache (append, read, attention), of the norms around
a residual sum and of the mixture-of-experts layer of a few tokens (include/awq.h).  Argument marshalling
only, as in _layer.py: one expression tests what a correct call satisfies, and only if it is false are
the arguments looked at one by one for the message."""
from __future__ import annotations

import ctypes
import math

import torch

from ._binding import AWQ_OK, AwqError, Kv4Cache, _empty, _need, last_error, load_library
from ._layer import (_DTYPES, _dense_or_same, _device, _f32, _given, _half, _half_dtypes, _handle, _heads, _i32, _library, _ok,
                     _on_current, scratch)

NORMS = {"rms": 0, "layer": 1}


def awq_kv4_page_bytes(page_size, head_dim, group_size=128) -> int:
    """Bytes of one head's tokens of a page of a 4-bit cache, page_size * (head_dim + 8 * head_dim /
    group_size): a cache is a uint8 tensor [pages, heads, awq_kv4_page_bytes(...)] (host only)."""
    b = ctypes.c_size_t(0)
    _ok(load_library().awq_kv4_page_bytes(page_size, head_dim, group_size, ctypes.byref(b)))
    return b.value


def _kv4(cache, heads, dim, group_size, device):
    shape = cache.shape
    if not (cache.dtype is torch.uint8 and len(shape) == 3 and (heads is None or shape[1] == heads) and
            cache.get_device() == device and (cache.stride(2) == 1 or shape[2] <= 1)):
        if cache.dtype is not torch.uint8 or len(shape) != 3:
            raise ValueError(f"cache must be a uint8 tensor [pages, heads, bytes], got {cache.dtype} {tuple(shape)}")
        if heads is not None and shape[1] != heads:
            raise ValueError(f"cache must have {heads} heads, got shape {tuple(shape)}")
        _heads(cache, "cache", torch.uint8, shape, device)
    if group_size not in (32, 64, 128) or dim % group_size:
        raise ValueError(f"group_size must be 32, 64 or 128 and divide the head size, got {group_size} of {dim}")
    per = dim + 8 * dim // group_size  # bytes of a token
    page = shape[2] // per
    if page * per != shape[2] or page % 16 or page == 0:
        raise ValueError(f"cache's last dimension must hold a multiple of 16 tokens of {per} bytes, got {shape[2]} bytes")
    return Kv4Cache(cache.data_ptr(), shape[0], page, shape[1], dim, group_size, cache.stride(0), cache.stride(1))


def awq_rope_append_kv4(q, k, v, positions, table, cache, slots, group_size=128, interleaved=False, q_out=None, stream=None):
    """awq_rope_append to a 4-bit cache, a uint8 tensor [pages, heads, bytes] (awq_kv4_page_bytes; pages and
    heads strided by multiples of 16): every group_size (32, 64, 128) neighbouring elements of the rotated
    keys and of the values v become 4-bit codes, a scale and a minimum of the element type at slots int32 [T].
    A slot outside the cache (-1) keeps nothing.  positions and table None: nothing is rotated, and q may
    be None.  Returns the rotated queries."""
    dt, dev, ks = k.dtype, k.get_device(), k.shape
    if not (dt in _half_dtypes and dev == _device() and len(ks) == 3 and v.dtype is dt and v.shape == ks and v.get_device() == dev and
            k.stride(2) == 1 and v.stride(2) == 1 and slots.dtype is _i32 and slots.shape == ks[:1] and slots.is_contiguous() and
            slots.get_device() == dev):
        _half(k, "k")
        if len(ks) != 3:
            raise ValueError("k must be [tokens, heads, head_dim]")
        dev = _on_current(k, "k")
        _heads(k, "k", dt, ks, dev)
        _heads(v, "v", dt, ks, dev)
        _need(slots, "slots", _i32, ks[:1], dev)
    T, Hkv, D = ks
    Hq = qt = qh = 0
    if q is not None:
        if not (q.dtype is dt and q.dim() == 3 and q.shape[0] == T and q.shape[2] == D and q.get_device() == dev and q.stride(2) == 1):
            if q.dim() != 3:
                raise ValueError("q must be [tokens, heads, head_dim]")
            _heads(q, "q", dt, (T, q.shape[1], D), dev)
        Hq, qt, qh = q.shape[1], q.stride(0), q.stride(1)
        q_out = _empty((T, Hq, D), dt, dev, stream) if q_out is None else _dense_or_same(q_out, q, "q_out", dt, dev)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    last = rot = 0
    if table is None:
        if positions is not None:
            raise ValueError("positions need a table")
    else:
        if positions is None:
            raise ValueError("a table needs positions")
        if table.dim() != 2:
            raise ValueError("table must be [max_position, rotary_dim]")
        last, rot = table.shape
        _need(positions, "positions", _i32, (T,), dev)
        _need(table, "table", _f32, (last, rot), dev)
    c = _kv4(cache, Hkv, D, group_size, dev)
    st = _library().awq_rope_append_kv4(None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                        None if table is None else positions.data_ptr(), None if table is None else table.data_ptr(),
                                        T, Hq, Hkv, D, rot, last, qt, qh, k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                                        None if q is None else q_out.data_ptr(), c, slots.data_ptr(), 1 if interleaved else 0,
                                        _DTYPES[dt], _handle(stream, dev))
    if st != AWQ_OK:
        raise AwqError(st, last_error())
    return q_out


def awq_kv4_read(cache, slots, head_dim, group_size=128, dtype=torch.float16, out=None, stream=None):
    """The keys and values that a 4-bit cache holds at slots int32 [T], rounded once to dtype, the element
    type it was written with: (k, v) [T, heads, head_dim], or fills ``out``, a tuple of those two.  A slot
    outside the cache reads zero."""
    if dtype not in _half_dtypes:
        raise TypeError(f"dtype must be float16 or bfloat16, got {dtype}")
    dev = _on_current(slots, "slots")
    if slots.dim() != 1:
        raise ValueError("slots must have one dimension")
    _need(slots, "slots", _i32, slots.shape, dev)
    c = _kv4(cache, None, head_dim, group_size, dev)
    shape = (slots.shape[0], cache.shape[1], head_dim)
    if out is None:
        k, v = _empty(shape, dtype, dev, stream), _empty(shape, dtype, dev, stream)
    else:
        k, v = out
        _need(k, "k", dtype, shape, dev)
        _need(v, "v", dtype, shape, dev)
    st = _library().awq_kv4_read(c, slots.data_ptr(), shape[0], k.data_ptr(), v.data_ptr(), _DTYPES[dtype], _handle(stream, dev))
    if st != AWQ_OK:
        raise AwqError(st, last_error())
    return k, v


def awq_attention_kv4(q, cache, pages, lens, group_size=128, window=0, sinks=0, scale=None, out=None, stream=None, workspace=None):
    """Attention of the n newest tokens of B sequences over a 4-bit cache (awq_rope_append_kv4).

    q fp16 or bf16 [B, n, Hq, D] or [B, Hq, D] (n = 1), heads contiguous, the element type the cache was
    written with (D 64, 96, 128 or 256; Hq a multiple of the cache's heads); pages int32 [B, W]: each
    sequence's pages in order; lens int32 [B]: its tokens, the n new ones last (causal among themselves).
    window > 0: a token sees its window last keys, itself among them, and the first ``sinks`` of the sequence.
    scale defaults to 1 / sqrt(D).  Returns q's shape, dense.
    workspace: a uint8 device tensor of awq_attention_kv4_workspace_size bytes (default: this module's for
    the stream)."""
    dt, dev, qs = q.dtype, q.get_device(), q.shape
    if len(qs) == 4:
        B, n, Hq, D = qs
        sb, sn, sh, one = q.stride()
    elif len(qs) == 3:
        B, Hq, D = qs
        n, sn = 1, 0
        sb, sh, one = q.stride()
    else:
        raise ValueError("q must be [B, n, heads, head_dim] or [B, heads, head_dim]")
    ps = pages.shape
    if not (dt in _half_dtypes and dev == _device() and one == 1 and len(ps) == 2 and ps[0] == B and pages.dtype is _i32 and
            pages.get_device() == dev and (ps[1] <= 1 or pages.stride(1) == 1) and lens.dtype is _i32 and lens.shape == (B,) and
            lens.is_contiguous() and lens.get_device() == dev):
        _half(q, "q")
        dev = _on_current(q, "q")
        _heads(q, "q", dt, qs, dev)
        if len(ps) != 2 or pages.dtype is not _i32 or ps[0] != B:
            raise ValueError(f"pages must be an int32 [{B}, W] table, got {pages.dtype} {tuple(ps)}")
        if B:
            _heads(pages, "pages", _i32, ps, dev)
        _need(lens, "lens", _i32, (B,), dev)
    c = _kv4(cache, None, D, group_size, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _empty(qs, dt, dev, stream)
    else:
        _need(out, "out", dt, qs, dev)
    handle, lib = _handle(stream, dev), _library()
    if workspace is None:
        need = ctypes.c_size_t(0)
        _ok(lib.awq_attention_kv4_workspace_size(B, n, Hq, cache.shape[1], D, need))
        ws = scratch(dev, handle, need.value)
    else:
        ws = _given(workspace, dev, "q")
    with ws[3]:
        st = lib.awq_attention_kv4(q.data_ptr(), B, n, Hq, sb, sn, sh, c, pages.data_ptr(), ps[1], pages.stride(0), lens.data_ptr(),
                                   window or 0, sinks, scale, out.data_ptr(), _DTYPES[dt], ws[0], ws[1], handle)
    if st != AWQ_OK:
        raise AwqError(st, last_error())
    return out


def awq_attention_kv4_workspace_size(B, n, Hq, heads, D) -> int:
    """Bytes of workspace an awq_attention_kv4 call of these sizes needs (host only)."""
    b = ctypes.c_size_t(0)
    _ok(load_library().awq_attention_kv4_workspace_size(B, n, Hq, heads, D, ctypes.byref(b)))
    return b.value


def _row_stride(t, name, dt, shape, device):
    if not (t.dtype is dt and t.shape == shape and t.get_device() == device and (t.stride(1) == 1 or shape[1] <= 1)):
        _heads(t, name, dt, shape, device)
    return t.stride(0)


def awq_residual_norm(x, residual=None, weight=None, bias=None, post_weight=None, post_bias=None, gate=None, scale=1.0, eps=1e-6,
                      kind="rms", out=None, stream=None):
    """The norms before and after a block, around its residual sum (fp16 or bf16):

        t = norm(x) * post_weight + post_bias     (x itself where post_weight is None)
        h = residual + scale * gate * t           (residual None: 0; gate None: 1)
        y = norm(h) * weight + bias               (None where weight is None)

    x, residual [T, W], rows contiguous; gate [W] or [T, W]; weights and biases [W]; kind "rms" or "layer".
    Returns (h, y), dense, or fills ``out``, a tuple of those two; h may be residual and y may be x."""
    dt, dev, xs = x.dtype, x.get_device(), x.shape
    if not (dt in _half_dtypes and dev == _device() and len(xs) == 2 and (x.stride(1) == 1 or xs[1] <= 1)):
        _half(x, "x")
        if len(xs) != 2:
            raise ValueError("x must be [tokens, width]")
        dev = _on_current(x, "x")
        _heads(x, "x", dt, xs, dev)
    if kind not in NORMS:
        raise ValueError(f"kind must be 'rms' or 'layer', got {kind!r}")
    T, W = xs
    rs = 0 if residual is None else _row_stride(residual, "residual", dt, xs, dev)
    gs = 0
    if gate is not None:
        if gate.dim() == 1:
            _need(gate, "gate", dt, (W,), dev)
        else:
            gs = _row_stride(gate, "gate", dt, xs, dev)
    for t, name in ((weight, "weight"), (bias, "bias"), (post_weight, "post_weight"), (post_bias, "post_bias")):
        if t is not None:
            _need(t, name, dt, (W,), dev)
    if out is None:
        h, y = _empty((T, W), dt, dev, stream), None if weight is None else _empty((T, W), dt, dev, stream)
    else:
        h, y = out
        _need(h, "h", dt, xs, dev)
        if weight is not None:
            _need(y, "y", dt, xs, dev)
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    st = _library().awq_residual_norm(x.data_ptr(), x.stride(0), at(residual), rs, at(gate), gs, at(post_weight), at(post_bias), scale,
                                      at(weight), at(bias), T, W, NORMS[kind], eps, h.data_ptr(),
                                      None if weight is None else y.data_ptr(), _DTYPES[dt], _handle(stream, dev))
    if st != AWQ_OK:
        raise AwqError(st, last_error())
    return h, y


def _stacked(linear, name, dt, E, K, N, group, device):
    qweight, qzeros, scales = linear
    _need(qweight, f"{name} qweight", _i32, (E, K, N // 8), device)
    _need(qzeros, f"{name} qzeros", _i32, (E, K // group, N // 8), device)
    _need(scales, f"{name} scales", dt, (E, K // group, N), device)
    return qweight.data_ptr(), qzeros.data_ptr(), scales.data_ptr()


def awq_moe_layer(x, weights, experts, up, down, group_size=128, base=None, out=None, stream=None, workspace=None):
    """A mixture-of-experts layer of at most 16 tokens on 4-bit experts, in two launches:

        out[t] = base[t] + sum_j weights[t, j] * (silu(x[t] gate) * (x[t] up)) down     of expert experts[t, j]

    x fp16 or bf16 [T, H], rows contiguous; (weights fp32, experts int32) [T, k] of awq_moe_route; up and down:
    (qweight, qzeros, scales) of the stacked experts, [E, H, 2 I / 8] ... with an expert's gate columns in
    front of its up columns, and [E, I, H / 8] ...; scales of x's type.  A place whose id lies outside [0, E)
    is left out.  base [T, H] or None; out may be base.  More tokens: awq_moe_dispatch, awq_gemm_grouped
    and awq_moe_combine.  workspace: a uint8 device tensor of awq_moe_layer_workspace_size bytes (default:
    the package's for the stream)."""
    dt, dev, xs, es = x.dtype, x.get_device(), x.shape, experts.shape
    if not (dt in _half_dtypes and dev == _device() and len(xs) == 2 and len(es) == 2 and es[0] == xs[0] and
            (x.stride(1) == 1 or xs[1] <= 1) and experts.dtype is _i32 and experts.is_contiguous() and experts.get_device() == dev and
            weights.dtype is _f32 and weights.shape == es and weights.is_contiguous() and weights.get_device() == dev):
        _half(x, "x")
        if len(xs) != 2 or len(es) != 2:
            raise ValueError("x must be [tokens, hidden], experts [tokens, k]")
        dev = _on_current(x, "x")
        _heads(x, "x", dt, xs, dev)
        _need(experts, "experts", _i32, (xs[0], es[1]), dev)
        _need(weights, "weights", _f32, es, dev)
    (T, H), k = xs, es[1]
    if group_size <= 0:
        raise ValueError(f"group_size must be positive, got {group_size}")
    if up[2].dim() != 3:
        raise ValueError("up scales must be [experts, hidden / group_size, 2 * inner]")
    E, I = up[2].shape[0], up[2].shape[2] // 2
    upp = _stacked(up, "up", dt, E, H, 2 * I, group_size, dev)
    downp = _stacked(down, "down", dt, E, I, H, group_size, dev)
    if base is not None:
        _need(base, "base", dt, xs, dev)
    if out is None:
        out = _empty(xs, dt, dev, stream)
    else:
        _need(out, "out", dt, xs, dev)
    handle, lib = _handle(stream, dev), _library()
    if workspace is None:
        need = ctypes.c_size_t(0)
        _ok(lib.awq_moe_layer_workspace_size(T, k, H, I, need))
        ws = scratch(dev, handle, need.value)
    else:
        ws = _given(workspace, dev, "x")
    with ws[3]:
        st = lib.awq_moe_layer(x.data_ptr(), T, H, x.stride(0), experts.data_ptr(), weights.data_ptr(), k, E, I, group_size, *upp,
                               *downp, None if base is None else base.data_ptr(), out.data_ptr(), _DTYPES[dt], ws[0], ws[1], handle)
    if st != AWQ_OK:
        raise AwqError(st, last_error())
    return out


def awq_moe_layer_workspace_size(T, k, H, I) -> int:
    """Bytes of workspace an awq_moe_layer call of these sizes needs (host only)."""
    b = ctypes.c_size_t(0)
    _ok(load_library().awq_moe_layer_workspace_size(T, k, H, I, ctypes.byref(b)))
    return b.value
