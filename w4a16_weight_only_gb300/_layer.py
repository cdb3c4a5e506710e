"""Binding of the operators between a decoder layer's linears (include/awq.h): rotary positions,
attention over a paged cache with a shared prefix, expert routing, dispatch and combine.  Argument
marshalling only, as in _binding.py: every step of the computation runs in the library's kernels."""
from __future__ import annotations

import ctypes
import math

import torch

from ._binding import (AWQ_OK, DTYPE_BF16, DTYPE_F16, DTYPE_F32, AwqError, PagedKV, _cuda_index, _need, last_error,
                       load_library)

ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "banded": 4}
_DTYPES = {torch.float16: DTYPE_F16, torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}
_GRANULE = 1 << 20

_scratch = {}


def _handle(stream, device):
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def scratch(device, handle, nbytes):
    """A uint8 workspace of at least ``nbytes`` that this module's calls on (device, stream) share:
    calls on one stream never overlap, and no call reads what an earlier one left.  It grows by
    allocation (at least doubling) and a smaller one is kept, since a captured CUDA graph may hold its
    address; make a stream's largest call once before capturing."""
    kept = _scratch.get((device, handle))
    if kept is None:
        kept = _scratch[(device, handle)] = []
    if not kept or kept[-1].numel() < nbytes:
        size = max(nbytes, 2 * kept[-1].numel() if kept else 0)
        kept.append(torch.empty(((size + _GRANULE - 1) // _GRANULE * _GRANULE,), dtype=torch.uint8, device=device))
    return kept[-1]


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
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, page_size, heads, head_dim]")
    shape = k_cache.shape
    if (heads is not None and shape[2] != heads) or shape[3] != dim:
        raise ValueError(f"k_cache must have {heads if heads is not None else 'some'} heads of {dim} elements, "
                         f"got shape {tuple(shape)}")
    _heads(k_cache, "k_cache", dt, shape, device)
    _heads(v_cache, "v_cache", dt, shape, device)
    s = k_cache.stride()
    if v_cache.stride() != s:
        raise ValueError("k_cache and v_cache must have the same strides")
    return PagedKV(k_cache.data_ptr(), v_cache.data_ptr(), shape[0], shape[1], shape[2], shape[3], s[0], s[1], s[2])


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
        out = torch.empty((max_position, rotary_dim), dtype=torch.float32, device="cuda" if device is None else device)
    dev = _cuda_index(out, "out")
    _need(out, "out", torch.float32, (max_position, rotary_dim), dev)
    p0, p1 = (low_factor, high_factor) if scaling == "banded" else (beta_fast, beta_slow)
    _ok(load_library().awq_rope_table(out.data_ptr(), max_position, rotary_dim, base, ROPE_SCALINGS[scaling], factor,
                                      original_max_position, p0, p1, attention_factor, _handle(stream, dev)))
    return out


def _rope_inputs(q, k, positions, table):
    dt, dev = _half(q, "q"), _cuda_index(q, "q")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    _heads(q, "q", dt, (T, Hq, D), dev)
    _heads(k, "k", dt, (T, Hkv, D), dev)
    _need(positions, "positions", torch.int32, (T,), dev)
    if table.dim() != 2:
        raise ValueError("table must be [max_position, rotary_dim]")
    _need(table, "table", torch.float32, table.shape, dev)
    return dt, dev, T, Hq, Hkv, D


def _dense_or_same(out, t, name, dt, dev):
    if out is None:
        return torch.empty(t.shape, dtype=dt, device=t.device)
    if out.data_ptr() == t.data_ptr() and out.stride() == t.stride() and out.shape == t.shape and out.dtype is dt:
        return out  # in place
    _need(out, name, dt, t.shape, dev)
    return out


def awq_rope(q, k, positions, table, interleaved=False, q_out=None, k_out=None, stream=None):
    """Rotates the first table.shape[1] elements of every head of q [T, Hq, D] and k [T, Hkv, D] (fp16
    or bf16; heads contiguous, other strides free) by the angles of positions int32 [T] and copies the
    rest.  Pairs are (i, i + rotary_dim / 2), or (2 i, 2 i + 1) with interleaved=True.  Returns
    (q_out, k_out), dense, or written in place where q_out is q (k_out is k)."""
    dt, dev, T, Hq, Hkv, D = _rope_inputs(q, k, positions, table)
    q_out = _dense_or_same(q_out, q, "q_out", dt, dev)
    k_out = _dense_or_same(k_out, k, "k_out", dt, dev)
    qs, ks = q.stride(), k.stride()
    _ok(load_library().awq_rope(q.data_ptr(), k.data_ptr(), positions.data_ptr(), table.data_ptr(), T, Hq, Hkv, D,
                                table.shape[1], table.shape[0], qs[0], qs[1], ks[0], ks[1], q_out.data_ptr(),
                                k_out.data_ptr(), 1 if interleaved else 0, _DTYPES[dt], _handle(stream, dev)))
    return q_out, k_out


def awq_rope_append(q, k, v, positions, table, k_cache, v_cache, slots, interleaved=False, q_out=None, stream=None):
    """awq_rope with the rotated keys, and the values v [T, Hkv, D], written to the paged cache (k_cache
    and v_cache [pages, page_size, Hkv, D], any equal strides with contiguous heads) at slots int32
    [T]: slot s is token s % page_size of page s // page_size, and a slot outside the cache (-1) keeps
    nothing.  Returns the rotated queries."""
    dt, dev, T, Hq, Hkv, D = _rope_inputs(q, k, positions, table)
    _heads(v, "v", dt, (T, Hkv, D), dev)
    _need(slots, "slots", torch.int32, (T,), dev)
    cache = _cache(k_cache, v_cache, dt, Hkv, D, dev)
    q_out = _dense_or_same(q_out, q, "q_out", dt, dev)
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    _ok(load_library().awq_rope_append(q.data_ptr(), k.data_ptr(), v.data_ptr(), positions.data_ptr(), table.data_ptr(), T,
                                       Hq, Hkv, D, table.shape[1], table.shape[0], qs[0], qs[1], ks[0], ks[1], vs[0], vs[1],
                                       q_out.data_ptr(), ctypes.byref(cache), slots.data_ptr(), 1 if interleaved else 0,
                                       _DTYPES[dt], _handle(stream, dev)))
    return q_out


def awq_attention_shared(q, k_cache, v_cache, prefix_pages, prefix_len, pages, lens, scale=None, max_len=None, out=None,
                         stream=None, workspace=None):
    """Attention of the n newest tokens of B sequences over a prefix that all share and their own keys.

    q fp16 or bf16 [B, n, Hq, D] or [B, Hq, D] (n = 1), heads contiguous; k_cache and v_cache [pages,
    page_size, heads, D] (D 64, 96, 128 or 256; Hq a multiple of heads), equal strides; prefix_pages
    int32 [>= ceil(prefix_len / page_size)]; pages int32 [B, W]; lens int32 [B]: own tokens of each
    sequence, the n new ones last (causal among themselves).  prefix_len and max_len (>= every length;
    default W * page_size) are host integers.  scale defaults to 1 / sqrt(D).  Returns q's shape, dense.
    workspace: a uint8 device tensor of awq_attention_shared_workspace_size bytes (default: this
    module's for the stream)."""
    lib = load_library()
    dt, dev = _half(q, "q"), _cuda_index(q, "q")
    if q.dim() == 3:
        B, Hq, D = q.shape
        n, sb, sn, sh = 1, q.stride(0), 0, q.stride(1)
    elif q.dim() == 4:
        B, n, Hq, D = q.shape
        sb, sn, sh = q.stride(0), q.stride(1), q.stride(2)
    else:
        raise ValueError("q must be [B, n, heads, head_dim] or [B, heads, head_dim]")
    _heads(q, "q", dt, q.shape, dev)
    cache = _cache(k_cache, v_cache, dt, None, D, dev)
    page = cache.page_size
    if prefix_pages.dim() != 1 or (page > 0 and prefix_pages.shape[0] * page < prefix_len):
        raise ValueError(f"prefix_pages must hold the pages of {prefix_len} tokens")
    _need(prefix_pages, "prefix_pages", torch.int32, prefix_pages.shape, dev)
    if pages.dim() != 2 or pages.dtype is not torch.int32 or pages.shape[0] != B:
        raise ValueError(f"pages must be an int32 [{B}, W] table, got {pages.dtype} {tuple(pages.shape)}")
    _heads(pages, "pages", torch.int32, pages.shape, dev)
    _need(lens, "lens", torch.int32, (B,), dev)
    if max_len is None:
        max_len = pages.shape[1] * page
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty(q.shape, dtype=dt, device=q.device)
    else:
        _need(out, "out", dt, q.shape, dev)
    handle = _handle(stream, dev)
    if workspace is None:
        workspace = scratch(dev, handle, awq_attention_shared_workspace_size(B, n, Hq, cache.heads, D, prefix_len, max_len))
    elif workspace.dtype is not torch.uint8 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on q's device")
    _ok(lib.awq_attention_shared(q.data_ptr(), B, n, Hq, sb, sn, sh, ctypes.byref(cache), prefix_pages.data_ptr(), prefix_len,
                                 pages.data_ptr(), pages.shape[1], pages.stride(0), lens.data_ptr(), max_len, scale,
                                 out.data_ptr(), _DTYPES[dt], workspace.data_ptr(), workspace.numel(), handle))
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
    if logits.dtype not in _DTYPES:
        raise TypeError(f"logits must be float16, bfloat16 or float32, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must be [tokens, experts]")
    if scoring not in ("softmax", "sigmoid"):
        raise ValueError(f"scoring must be 'softmax' or 'sigmoid', got {scoring!r}")
    dev = _cuda_index(logits, "logits")
    T, E = logits.shape
    _heads(logits, "logits", logits.dtype, (T, E), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, (E,), dev)
    if out is None:
        weights = torch.empty((T, topk), dtype=torch.float32, device=logits.device)
        experts = torch.empty((T, topk), dtype=torch.int32, device=logits.device)
    else:
        weights, experts = out
        _need(weights, "weights", torch.float32, (T, topk), dev)
        _need(experts, "experts", torch.int32, (T, topk), dev)
    _ok(load_library().awq_moe_route(logits.data_ptr(), T, E, logits.stride(0), _DTYPES[logits.dtype], topk,
                                     1 if scoring == "sigmoid" else 0, None if bias is None else bias.data_ptr(), groups,
                                     topk_groups, group_best, 1 if renormalize else 0, scale, weights.data_ptr(),
                                     experts.data_ptr(), _handle(stream, dev)))
    return weights, experts


def awq_moe_dispatch(x, experts, num_experts, out=None, stream=None, workspace=None):
    """Sorts the places of experts int32 [T, k] by expert and gathers the rows of x [T, W] (fp16 or
    bf16, rows contiguous) accordingly: what awq_gemm_grouped and awq_gemm_packed_grouped take.  Returns
    (routed [T k, W], offsets int32 [num_experts + 1], rows int32 [T, k]: each place's row), or fills
    ``out``, a tuple of those three.  A place whose id lies outside [0, num_experts) gets row -1; the
    rows of routed behind offsets[-1] are zero.  workspace: a uint8 device tensor of
    awq_moe_dispatch_workspace_size bytes (default: this module's for the stream)."""
    lib = load_library()
    dt, dev = _half(x, "x"), _cuda_index(x, "x")
    if x.dim() != 2 or experts.dim() != 2:
        raise ValueError("x must be [tokens, width], experts [tokens, k]")
    T, W = x.shape
    k = experts.shape[1]
    _heads(x, "x", dt, (T, W), dev)
    _need(experts, "experts", torch.int32, (T, k), dev)
    if out is None:
        routed = torch.empty((T * k, W), dtype=dt, device=x.device)
        offsets = torch.empty((num_experts + 1,), dtype=torch.int32, device=x.device)
        rows = torch.empty((T, k), dtype=torch.int32, device=x.device)
    else:
        routed, offsets, rows = out
        _need(routed, "routed", dt, (T * k, W), dev)
        _need(offsets, "offsets", torch.int32, (num_experts + 1,), dev)
        _need(rows, "rows", torch.int32, (T, k), dev)
    handle = _handle(stream, dev)
    if workspace is None:
        workspace = scratch(dev, handle, awq_moe_dispatch_workspace_size(T, k, num_experts))
    elif workspace.dtype is not torch.uint8 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on x's device")
    _ok(lib.awq_moe_dispatch(x.data_ptr(), T, W, x.stride(0), experts.data_ptr(), k, num_experts, routed.data_ptr(),
                             offsets.data_ptr(), rows.data_ptr(), workspace.data_ptr(), workspace.numel(), handle))
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
    dt, dev = _half(y, "y"), _cuda_index(y, "y")
    if y.dim() != 2 or rows.dim() != 2:
        raise ValueError("y must be [rows, width], rows [tokens, k]")
    R, W = y.shape
    T, k = rows.shape
    _need(y, "y", dt, (R, W), dev)
    _need(weights, "weights", torch.float32, (T, k), dev)
    _need(rows, "rows", torch.int32, (T, k), dev)
    if base is not None:
        _need(base, "base", dt, (T, W), dev)
    if out is None:
        out = torch.empty((T, W), dtype=dt, device=y.device)
    else:
        _need(out, "out", dt, (T, W), dev)
    _ok(load_library().awq_moe_combine(y.data_ptr(), R, W, weights.data_ptr(), rows.data_ptr(), T, k,
                                       None if base is None else base.data_ptr(), out.data_ptr(), _DTYPES[dt],
                                       _handle(stream, dev)))
    return out
