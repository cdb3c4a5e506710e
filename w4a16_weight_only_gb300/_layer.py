"""Binding of the operators between a decoder layer's linears (include/awq.h): rotary positions,
attention over a paged cache with a shared prefix, expert routing, dispatch and combine.  Argument
marshalling only, as in _binding.py: every step of the computation runs in the library's kernels."""
from __future__ import annotations

import contextlib
import ctypes
import math
import threading

import torch

from . import _binding
from ._binding import (AWQ_OK, DTYPE_BF16, DTYPE_F16, DTYPE_F32, AwqError, PagedKV, _allocating_for, _cuda_index, _current,
                       _empty, _need, last_error, load_library)

ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "banded": 4}
_DTYPES = {torch.float16: DTYPE_F16, torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}
_GRANULE = 1 << 20

_scratch = {}


# The calls below run once per layer and token, so they are written for few interpreter steps: one
# expression tests what a correct call satisfies, and only if it is false are the arguments looked at
# one by one for the message (17 and 24 us of host time for awq_rope_append and awq_attention_shared;
# 19 and 28 with a helper call per tensor).
_half_dtypes = (torch.float16, torch.bfloat16)
_i32, _f32 = torch.int32, torch.float32


# torch.cuda.current_device() without its check that CUDA is up: a tensor of it exists where this is asked
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on_current(t, name):
    """The device of a CUDA tensor, which has to be the current one: that is where the library launches."""
    dev = _cuda_index(t, name)
    if dev != _device():
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{_device()}: call under torch.cuda.device")
    return dev


def _handle(stream, device):
    if stream is None:
        return _current(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _library():
    return _binding._lib or load_library()


def scratch(device, handle, nbytes):
    """(address, bytes, tensor, lock) of a workspace of at least ``nbytes`` that this module's calls on
    (device, stream) share: kernels of one stream run in the order of their launches, and no call reads
    what an earlier one left.  A call of several launches holds the lock while it enqueues them, since
    another host thread's launches on the stream must not come between.  The workspace grows by
    allocation (at least doubling) and a smaller one is kept, since a captured CUDA graph may hold its
    address; make a stream's largest call once before capturing.  A graph keeps the workspace of the
    stream that captured it: replayed beside other calls of that stream, it needs a workspace of its own."""
    lock, kept = _scratch.get((device, handle)) or _scratch.setdefault((device, handle), (threading.Lock(), []))
    with lock:
        if not kept or kept[-1][1] < nbytes:
            size = (max(nbytes, 2 * kept[-1][1] if kept else 0) + _GRANULE - 1) // _GRANULE * _GRANULE
            with _allocating_for(handle, device):
                t = torch.empty((size,), dtype=torch.uint8, device=device)
            kept.append((t.data_ptr(), size, t, lock))
        return kept[-1]


_no_lock = contextlib.nullcontext()  # calls that share a workspace given by the caller: the caller keeps them apart


def _given(workspace, device, name):
    if workspace.dtype is not torch.uint8 or workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {name}'s device")
    return workspace.data_ptr(), workspace.numel(), workspace, _no_lock


def _half(t, name):
    dt = t.dtype
    if dt is not torch.float16 and dt is not torch.bfloat16:
        raise TypeError(f"{name} must be float16 or bfloat16, got {dt}")
    return dt


def _heads(t, name, dt, shape, device):
    """Like _need for a tensor whose last dimension alone has to be contiguous."""
    if t.dtype is not dt:
        raise TypeError(f"{name} must be {dt}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected device {device}")
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _cache(k_cache, v_cache, dt, heads, dim, device):
    shape, s = k_cache.shape, k_cache.stride()
    if not (len(shape) == 4 and (heads is None or shape[2] == heads) and shape[3] == dim and k_cache.dtype is dt and
            v_cache.dtype is dt and v_cache.shape == shape and v_cache.stride() == s and k_cache.get_device() == device and
            v_cache.get_device() == device and s[3] == 1):
        if len(shape) != 4:
            raise ValueError("k_cache must be [pages, page_size, heads, head_dim]")
        if (heads is not None and shape[2] != heads) or shape[3] != dim:
            raise ValueError(f"k_cache must have {heads if heads is not None else 'some'} heads of {dim} elements, "
                             f"got shape {tuple(shape)}")
        _heads(k_cache, "k_cache", dt, shape, device)
        _heads(v_cache, "v_cache", dt, shape, device)
        if any(a != b for a, b, size in zip(v_cache.stride(), s, shape) if size > 1):
            raise ValueError("k_cache and v_cache must have the same strides")
    return PagedKV(k_cache.data_ptr(), v_cache.data_ptr(), *shape, s[0], s[1], s[2])


def _ok(status):
    if status != AWQ_OK:
        raise AwqError(status, last_error())


def awq_rope_table(max_position, rotary_dim, base=10000.0, scaling="none", factor=1.0, original_max_position=0,
                   beta_fast=32.0, beta_slow=1.0, low_factor=1.0, high_factor=4.0, attention_factor=None, device=None,
                   out=None, stream=None):
    """The fp32 table [max_position, rotary_dim] (cosines, then sines, of every pair) that awq_rope
    reads; angles are formed in 64 bits.  scaling: "none", "linear", "ntk", "yarn" (beta_fast,
    beta_slow) or "banded" (low_factor, high_factor), for contexts ``factor`` times
    original_max_position; attention_factor multiplies cosines and sines (default 1; "yarn":
    0.1 ln(factor) + 1)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    if attention_factor is None:
        attention_factor = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1 else 1.0
    if out is None:
        where = torch.device("cuda" if device is None else device)
        if where.type != "cuda":
            raise ValueError(f"device must be a CUDA device, got {where}")
        out = _empty((max_position, rotary_dim), _f32, torch.cuda.current_device() if where.index is None else where.index, stream)
    dev = _on_current(out, "out")
    _need(out, "out", torch.float32, (max_position, rotary_dim), dev)
    p0, p1 = (low_factor, high_factor) if scaling == "banded" else (beta_fast, beta_slow)
    _ok(load_library().awq_rope_table(out.data_ptr(), max_position, rotary_dim, base, ROPE_SCALINGS[scaling], factor,
                                      original_max_position, p0, p1, attention_factor, _handle(stream, dev)))
    return out


def _rope_inputs(q, k, positions, table):
    dt, dev = q.dtype, q.get_device()
    qs, ks, ts = q.shape, k.shape, table.shape
    if not (dt in _half_dtypes and dev == _device() and len(qs) == 3 and len(ks) == 3 and len(ts) == 2 and k.dtype is dt and
            ks[0] == qs[0] and ks[2] == qs[2] and k.get_device() == dev and positions.dtype is _i32 and
            positions.shape == qs[:1] and positions.is_contiguous() and positions.get_device() == dev and
            table.dtype is _f32 and table.is_contiguous() and table.get_device() == dev and
            (qs[2] <= 1 or (q.stride(2) == 1 and k.stride(2) == 1))):
        _half(q, "q")
        dev = _on_current(q, "q")
        if len(qs) != 3 or len(ks) != 3:
            raise ValueError("q and k must be [tokens, heads, head_dim]")
        if len(ts) != 2:
            raise ValueError("table must be [max_position, rotary_dim]")
        _heads(q, "q", dt, qs, dev)
        _heads(k, "k", dt, (qs[0], ks[1], qs[2]), dev)
        _need(positions, "positions", _i32, (qs[0],), dev)
        _need(table, "table", _f32, ts, dev)
    return dt, dev, qs, ks[1], ts


def _dense_or_same(out, t, name, dt, dev):
    if out.data_ptr() == t.data_ptr() and out.stride() == t.stride() and out.shape == t.shape and out.dtype is dt:
        return out  # in place
    if out.numel() and out.data_ptr() == t.data_ptr():
        raise ValueError(f"{name} starts where its input does but has other strides")
    _need(out, name, dt, t.shape, dev)
    return out


def awq_rope(q, k, positions, table, interleaved=False, q_out=None, k_out=None, stream=None):
    """Rotates the first table.shape[1] elements of every head of q [T, Hq, D] and k [T, Hkv, D] (fp16
    or bf16; heads contiguous, other strides free) by the angles of positions int32 [T] and copies the
    rest.  Pairs are (i, i + rotary_dim / 2), or (2 i, 2 i + 1) with interleaved=True.  Returns
    (q_out, k_out), dense, or written in place where q_out is q (k_out is k)."""
    dt, dev, (T, Hq, D), Hkv, (last, rot) = _rope_inputs(q, k, positions, table)
    q_out = _empty((T, Hq, D), dt, dev, stream) if q_out is None else _dense_or_same(q_out, q, "q_out", dt, dev)
    k_out = _empty((T, Hkv, D), dt, dev, stream) if k_out is None else _dense_or_same(k_out, k, "k_out", dt, dev)
    st = _library().awq_rope(q.data_ptr(), k.data_ptr(), positions.data_ptr(), table.data_ptr(), T, Hq, Hkv, D, rot, last,
                             q.stride(0), q.stride(1), k.stride(0), k.stride(1), q_out.data_ptr(), k_out.data_ptr(),
                             1 if interleaved else 0, _DTYPES[dt], _handle(stream, dev))
    if st != AWQ_OK:
        raise AwqError(st, last_error())
    return q_out, k_out


def awq_rope_append(q, k, v, positions, table, k_cache, v_cache, slots, interleaved=False, q_out=None, stream=None):
    """awq_rope with the rotated keys, and the values v [T, Hkv, D], written to the paged cache (k_cache
    and v_cache [pages, page_size, Hkv, D], any equal strides with contiguous heads) at slots int32
    [T]: slot s is token s % page_size of page s // page_size, and a slot outside the cache (-1) keeps
    nothing.  Returns the rotated queries."""
    dt, dev, (T, Hq, D), Hkv, (last, rot) = _rope_inputs(q, k, positions, table)
    if not (v.dtype is dt and v.shape == k.shape and v.get_device() == dev and (D <= 1 or v.stride(2) == 1) and
            slots.dtype is _i32 and slots.shape == (T,) and slots.is_contiguous() and slots.get_device() == dev):
        _heads(v, "v", dt, (T, Hkv, D), dev)
        _need(slots, "slots", _i32, (T,), dev)
    cache = _cache(k_cache, v_cache, dt, Hkv, D, dev)
    q_out = _empty((T, Hq, D), dt, dev, stream) if q_out is None else _dense_or_same(q_out, q, "q_out", dt, dev)
    st = _library().awq_rope_append(q.data_ptr(), k.data_ptr(), v.data_ptr(), positions.data_ptr(), table.data_ptr(), T, Hq,
                                    Hkv, D, rot, last, q.stride(0), q.stride(1), k.stride(0), k.stride(1), v.stride(0),
                                    v.stride(1), q_out.data_ptr(), cache, slots.data_ptr(), 1 if interleaved else 0,
                                    _DTYPES[dt], _handle(stream, dev))
    if st != AWQ_OK:
        raise AwqError(st, last_error())
    return q_out


def awq_attention_shared(q, k_cache, v_cache, prefix_pages, prefix_len, pages, lens, scale=None, max_len=None, out=None,
                         stream=None, workspace=None):
    """Attention of the n newest tokens of B sequences over a prefix that all share and their own keys.

    q fp16 or bf16 [B, n, Hq, D] or [B, Hq, D] (n = 1), heads contiguous; k_cache and v_cache [pages,
    page_size, heads, D] (D 64, 96, 128 or 256; Hq a multiple of heads), equal strides; prefix_pages
    int32 [>= ceil(prefix_len / page_size)]; pages int32 [B, W]; lens int32 [B]: own tokens of each
    sequence, the n new ones last (causal among themselves).  prefix_len and max_len (>= every length;
    default W * page_size) are host integers; pass a max_len near the longest length where the table is
    much wider: far above four times the average length the call slows down with it (awq.h).  scale
    defaults to 1 / sqrt(D).  Returns q's shape, dense.
    workspace: a uint8 device tensor of awq_attention_shared_workspace_size bytes (default: this
    module's for the stream)."""
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
            pages.get_device() == dev and (ps[1] <= 1 or pages.stride(1) == 1) and prefix_pages.dtype is _i32 and
            prefix_pages.dim() == 1 and prefix_pages.is_contiguous() and prefix_pages.get_device() == dev and
            lens.dtype is _i32 and lens.shape == (B,) and lens.is_contiguous() and lens.get_device() == dev):
        _half(q, "q")
        dev = _on_current(q, "q")
        _heads(q, "q", dt, qs, dev)
        if len(ps) != 2 or pages.dtype is not _i32 or ps[0] != B:
            raise ValueError(f"pages must be an int32 [{B}, W] table, got {pages.dtype} {tuple(ps)}")
        if B:
            _heads(pages, "pages", _i32, ps, dev)
        if prefix_pages.dim() != 1:
            raise ValueError("prefix_pages must have one dimension")
        _need(prefix_pages, "prefix_pages", _i32, prefix_pages.shape, dev)
        _need(lens, "lens", _i32, (B,), dev)
    cache = _cache(k_cache, v_cache, dt, None, D, dev)
    page, heads = k_cache.shape[1:3]
    if page > 0 and prefix_pages.shape[0] * page < prefix_len:
        raise ValueError(f"prefix_pages must hold the pages of {prefix_len} tokens")
    if max_len is None:
        max_len = ps[1] * page
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _empty(qs, dt, dev, stream)
    else:
        _need(out, "out", dt, qs, dev)
    handle, lib = _handle(stream, dev), _library()
    need = ctypes.c_size_t(0)
    if workspace is None:
        _ok(lib.awq_attention_shared_workspace_size(B, n, Hq, heads, D, prefix_len, max_len, need))
        ws = scratch(dev, handle, need.value)
    else:
        ws = _given(workspace, dev, "q")
    with ws[3]:
        st = lib.awq_attention_shared(q.data_ptr(), B, n, Hq, sb, sn, sh, cache, prefix_pages.data_ptr(), prefix_len,
                                      pages.data_ptr(), ps[1], pages.stride(0), lens.data_ptr(), max_len, scale,
                                      out.data_ptr(), _DTYPES[dt], ws[0], ws[1], handle)
    if st != AWQ_OK:
        raise AwqError(st, last_error())
    return out


def awq_attention_shared_workspace_size(B, n, Hq, heads, D, prefix_len, max_len) -> int:
    """Bytes of workspace an awq_attention_shared call of these sizes needs (host only)."""
    b = ctypes.c_size_t(0)
    _ok(load_library().awq_attention_shared_workspace_size(B, n, Hq, heads, D, prefix_len, max_len, ctypes.byref(b)))
    return b.value


def awq_moe_route(logits, topk, scoring="softmax", bias=None, groups=1, topk_groups=1, group_best=1, renormalize=True,
                  scale=1.0, out=None, stream=None):
    """The topk experts of each row of logits [T, E] (fp16, bf16 or fp32; rows contiguous) and their
    weights: scores by "softmax" or "sigmoid", ranked with an optional bias fp32 [E] within the
    topk_groups best of ``groups`` groups (a group's score: the sum of its group_best best keys), the
    scores divided by their sum if renormalize, times scale.  Equal keys go to the lower index.  Returns
    (weights fp32 [T, topk], experts int32 [T, topk]), or fills ``out``, a tuple of those two."""
    dt, dev, shape = logits.dtype, logits.get_device(), logits.shape
    if not (dt in _DTYPES and len(shape) == 2 and dev == _device() and (logits.stride(1) == 1 or shape[1] <= 1) and
            scoring in ("softmax", "sigmoid")):
        if dt not in _DTYPES:
            raise TypeError(f"logits must be float16, bfloat16 or float32, got {dt}")
        if len(shape) != 2:
            raise ValueError("logits must be [tokens, experts]")
        if scoring not in ("softmax", "sigmoid"):
            raise ValueError(f"scoring must be 'softmax' or 'sigmoid', got {scoring!r}")
        _heads(logits, "logits", dt, shape, _on_current(logits, "logits"))
    T, E = shape
    if bias is not None:
        _need(bias, "bias", _f32, (E,), dev)
    if out is None:
        weights = _empty((T, topk), _f32, dev, stream)
        experts = _empty((T, topk), _i32, dev, stream)
    else:
        weights, experts = out
        _need(weights, "weights", _f32, (T, topk), dev)
        _need(experts, "experts", _i32, (T, topk), dev)
    st = _library().awq_moe_route(logits.data_ptr(), T, E, logits.stride(0), _DTYPES[dt], topk,
                                  1 if scoring == "sigmoid" else 0, None if bias is None else bias.data_ptr(), groups,
                                  topk_groups, group_best, 1 if renormalize else 0, scale, weights.data_ptr(),
                                  experts.data_ptr(), _handle(stream, dev))
    if st != AWQ_OK:
        raise AwqError(st, last_error())
    return weights, experts


def awq_moe_dispatch(x, experts, num_experts, out=None, stream=None, workspace=None):
    """Sorts the places of experts int32 [T, k] by expert and gathers the rows of x [T, W] (fp16 or
    bf16, rows contiguous) accordingly: what awq_gemm_grouped and awq_gemm_packed_grouped take.  Returns
    (routed [T k, W], offsets int32 [num_experts + 1], rows int32 [T, k]: each place's row), or fills
    ``out``, a tuple of those three.  A place whose id lies outside [0, num_experts) gets row -1; the
    rows of routed behind offsets[-1] are zero.  workspace: a uint8 device tensor of
    awq_moe_dispatch_workspace_size bytes (default: this module's for the stream)."""
    dt, dev, xs, es = x.dtype, x.get_device(), x.shape, experts.shape
    if not (dt in _half_dtypes and dev == _device() and len(xs) == 2 and len(es) == 2 and es[0] == xs[0] and
            (x.stride(1) == 1 or xs[1] <= 1) and experts.dtype is _i32 and experts.is_contiguous() and
            experts.get_device() == dev):
        _half(x, "x")
        if len(xs) != 2 or len(es) != 2:
            raise ValueError("x must be [tokens, width], experts [tokens, k]")
        dev = _on_current(x, "x")
        _heads(x, "x", dt, xs, dev)
        _need(experts, "experts", _i32, (xs[0], es[1]), dev)
    (T, W), k = xs, es[1]
    if out is None:
        routed = _empty((T * k, W), dt, dev, stream)
        offsets = _empty((num_experts + 1,), _i32, dev, stream)
        rows = _empty((T, k), _i32, dev, stream)
    else:
        routed, offsets, rows = out
        _need(routed, "routed", dt, (T * k, W), dev)
        _need(offsets, "offsets", _i32, (num_experts + 1,), dev)
        _need(rows, "rows", _i32, (T, k), dev)
    handle, lib = _handle(stream, dev), _library()
    if workspace is None:
        need = ctypes.c_size_t(0)
        _ok(lib.awq_moe_dispatch_workspace_size(T, k, num_experts, need))
        ws = scratch(dev, handle, need.value)
    else:
        ws = _given(workspace, dev, "x")
    with ws[3]:
        st = lib.awq_moe_dispatch(x.data_ptr(), T, W, x.stride(0), experts.data_ptr(), k, num_experts, routed.data_ptr(),
                                  offsets.data_ptr(), rows.data_ptr(), ws[0], ws[1], handle)
    if st != AWQ_OK:
        raise AwqError(st, last_error())
    return routed, offsets, rows


def awq_moe_dispatch_workspace_size(T, k, num_experts) -> int:
    """Bytes of workspace an awq_moe_dispatch call of these sizes needs (host only)."""
    b = ctypes.c_size_t(0)
    _ok(load_library().awq_moe_dispatch_workspace_size(T, k, num_experts, ctypes.byref(b)))
    return b.value


def awq_moe_combine(y, weights, rows, base=None, out=None, stream=None):
    """out[t] = base[t] + sum_j weights[t, j] * y[rows[t, j]], in fp32 in the order of the places: y [R,
    W] fp16 or bf16, weights fp32 [T, k], rows int32 [T, k] (outside [0, R): left out), base [T, W] or
    None.  Returns [T, W]; out may be base."""
    dt, dev, ys, rs = y.dtype, y.get_device(), y.shape, rows.shape
    if not (dt in _half_dtypes and dev == _device() and len(ys) == 2 and len(rs) == 2 and y.is_contiguous() and rows.dtype is _i32 and
            rows.is_contiguous() and rows.get_device() == dev and weights.dtype is _f32 and weights.shape == rs and
            weights.is_contiguous() and weights.get_device() == dev):
        _half(y, "y")
        if len(ys) != 2 or len(rs) != 2:
            raise ValueError("y must be [rows, width], rows [tokens, k]")
        dev = _on_current(y, "y")
        _need(y, "y", dt, ys, dev)
        _need(weights, "weights", _f32, rs, dev)
        _need(rows, "rows", _i32, rs, dev)
    (R, W), (T, k) = ys, rs
    if base is not None:
        _need(base, "base", dt, (T, W), dev)
    if out is None:
        out = _empty((T, W), dt, dev, stream)
    else:
        _need(out, "out", dt, (T, W), dev)
    st = _library().awq_moe_combine(y.data_ptr(), R, W, weights.data_ptr(), rows.data_ptr(), T, k,
                                    None if base is None else base.data_ptr(), out.data_ptr(), _DTYPES[dt],
                                    _handle(stream, dev))
    if st != AWQ_OK:
        raise AwqError(st, last_error())
    return out
