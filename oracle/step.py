"""Plain numpy restatements of the operators around a 4-bit key/value cache, of the norms around a residual
sum and of the mixture-of-experts layer of a few tokens.  Written from the formulas; shares no code with
the library.  Quantization follows the definition operation by operation in fp32; the others are in 64
bits and also return the magnitudes that bound an implementation's rounding errors."""
from __future__ import annotations

import numpy as np

ORDER = (0, 2, 4, 6, 1, 3, 5, 7)


def round_to(x, dtype):
    """fp32 values of fp32 or fp64 x rounded once (to nearest even) to "fp16" or "bf16"."""
    x = np.asarray(x, dtype=np.float32)
    if dtype == "fp16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16).astype(np.float32)
    bits = x.view(np.uint32).astype(np.uint64)
    up = ((bits + 0x7FFF + ((bits >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), x, up)


def rotate(x, positions, table, dtype, interleaved=False):
    """x [T, H, D] fp32 values of the element type, rotated with every operation rounded to fp32 and the
    result to the element type.  A position outside the table gives NaN."""
    x, table = np.asarray(x, dtype=np.float32), np.asarray(table, dtype=np.float32)
    y, half = x.copy(), table.shape[1] // 2
    for t, pos in enumerate(positions):
        line = table[pos] if 0 <= pos < table.shape[0] else np.full(2 * half, np.nan, dtype=np.float32)
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = line[i], line[half + i]
            y[t, :, a] = round_to(x[t, :, a] * c - x[t, :, b] * s, dtype)
            y[t, :, b] = round_to(x[t, :, b] * c + x[t, :, a] * s, dtype)
    return y


def quantize(x, group, dtype):
    """x [..., D] -> codes uint8 [..., D], scale and minimum fp32 values of the element type [..., D / group]."""
    x = np.asarray(x, dtype=np.float32)
    by = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    bad = ~np.isfinite(by).all(-1, keepdims=True)
    half = np.float32(0.5)
    with np.errstate(all="ignore"):
        low, high = by.min(-1, keepdims=True), by.max(-1, keepdims=True)
        scale = round_to((high * half - low * half) / np.float32(7.5), dtype)
        code = np.rint((by * half - low * half) / (scale * half)).clip(0, 15)
        code = np.where(~bad & (scale > 0), code, 0).astype(np.uint8)
    nan = np.float32(np.nan)
    return code.reshape(x.shape), np.where(bad, nan, scale)[..., 0], np.where(bad, nan, low)[..., 0]


def dequantize(code, scale, low):
    """What the codes stand for, in 64 bits."""
    by = code.reshape(*scale.shape, code.shape[-1] // scale.shape[-1]).astype(np.float64)
    return (by * np.asarray(scale, np.float64)[..., None] + np.asarray(low, np.float64)[..., None]).reshape(code.shape)


def element_bits(x, dtype):
    """16-bit patterns of fp32 values that the element type holds."""
    x = np.asarray(x, dtype=np.float32)
    return x.astype(np.float16).view(np.uint16) if dtype == "fp16" else (x.view(np.uint32) >> 16).astype(np.uint16)


def key_byte(D, r, e):
    """Byte of a tile that holds the code of element e of token r's key."""
    W, w, j = min(D, 128) // 32, e // 8, e % 8
    a, b, t = w // 16, w % 16 // 4, w % 4
    return 1024 * a + 16 * W * r + 4 * (W * t + b) + j // 2


def value_byte(D, r, e):
    u, g, j = e // 32, e % 32 // 4, e % 4
    h, t, o = r // 8, r % 8 // 2, r % 2
    if u == D // 32 - 1 and u % 2 == 0:
        return 8 * D + 512 * (u // 2) + 8 * (4 * g + t) + 4 * h + 2 * o + j // 2
    return 8 * D + 512 * (u // 2) + 16 * (4 * g + t) + 8 * (u % 2) + 4 * h + 2 * o + j // 2


def store(cache, page_size, slot, k, v, dtype):
    """Writes a token's quantized keys and values, (code [H, D], scale [H, G], minimum [H, G]) each, to cache uint8
    [pages, H, bytes] at a slot."""
    if not 0 <= slot < cache.shape[0] * page_size:
        return
    H, D = k[0].shape
    G = k[1].shape[1]
    page, token = divmod(slot, page_size)
    first, r = token // 16 * 16 * (D + 8 * G), token % 16
    for part, (code, scale, low), byte in ((0, k, key_byte), (1, v, value_byte)):
        for e in range(D):
            at = first + byte(D, r, e)
            shift = 4 * (e % 2)
            cache[page, :, at] = (cache[page, :, at] & (0xF0 >> shift)) | (code[:, e] << shift)
        pairs = np.stack([element_bits(scale, dtype), element_bits(low, dtype)], axis=-1)  # [H, G, 2]
        at = first + 16 * D + part * 64 * G + 4 * G * r
        cache[page, :, at:at + 4 * G] = np.ascontiguousarray(pairs).view(np.uint8).reshape(H, 4 * G)


def attention(q, keys, values, lens, scale, window=0, sinks=0):
    """q [B, n, Hq, D]; keys[b], values[b]: (what the codes stand for, code * scale + |minimum|), [tokens, heads, D].
    Returns (out, sum_j p_j (code * scale + |minimum|) of the values, largest scale * sum |q| (..) of the keys)."""
    B, n, Hq, D = q.shape
    out, spread, largest = np.zeros(q.shape), np.zeros(q.shape), 0.0
    for b in range(B):
        heads = keys[b][0].shape[1]
        for i in range(n):
            at = lens[b] - n + i
            seen = [j for j in range(at + 1) if window == 0 or j > at - window or j < sinks]
            if not seen:
                continue
            for h in range(Hq):
                hk, qh = h // (Hq // heads), q[b, i, h].astype(np.float64)
                z = scale * (keys[b][0][seen, hk] @ qh)
                largest = max(largest, float((abs(scale) * (keys[b][1][seen, hk] @ np.abs(qh))).max()))
                p = np.exp(z - z.max())
                p /= p.sum()
                out[b, i, h], spread[b, i, h] = p @ values[b][0][seen, hk], p @ values[b][1][seen, hk]
    return out, spread, largest


def residual_norm(x, residual=None, weight=None, bias=None, post_weight=None, post_bias=None, gate=None, scale=1.0, eps=1e-6,
                  kind="rms"):
    """(h, y, bound of h's fp32 error, bound of y's) in 64 bits."""
    W = x.shape[1]
    e = 2.0 ** -22 * (64 + W / 256)

    def norm(z, dz):
        """A norm's value and the error of an fp32 evaluation of z known to dz."""
        mean = z.mean(-1, keepdims=True) if kind == "layer" else 0.0
        centred = z - mean
        r = 1 / np.sqrt((centred ** 2).mean(-1, keepdims=True) + eps)
        size = np.abs(z) + np.abs(z).mean(-1, keepdims=True) * (kind == "layer")
        moved = dz + dz.mean(-1, keepdims=True) + e * size  # of an element of z - mean
        # the root's relative error: errors of z enter through sum(z dz) / sum(z^2), Cauchy-Schwarz
        rel = e + np.sqrt((moved ** 2).mean(-1, keepdims=True)) * r
        return centred * r, moved * r + rel * np.abs(centred * r)

    f = lambda a: np.asarray(a, dtype=np.float64)  # noqa: E731
    t, dt = f(x), np.zeros(x.shape)
    if post_weight is not None:
        t, dt = norm(t, dt)
        t, dt = t * f(post_weight), dt * np.abs(f(post_weight)) + e * np.abs(t * f(post_weight))
        if post_bias is not None:
            t = t + f(post_bias)
            dt = dt + 2.0 ** -23 * np.abs(t)
    if gate is not None:
        t, dt = t * f(gate), dt * np.abs(f(gate)) + 2.0 ** -23 * np.abs(t * f(gate))
    t, dt = scale * t, abs(scale) * dt + 2.0 ** -23 * np.abs(scale * t)
    h = t if residual is None else f(residual) + t
    dh = dt + 2.0 ** -23 * np.abs(h)
    if weight is None:
        return h, None, dh, None
    y, dy = norm(h, dh)
    y, dy = y * f(weight), dy * np.abs(f(weight)) + 2.0 ** -22 * np.abs(y * f(weight))
    if bias is not None:
        y = y + f(bias)
        dy = dy + 2.0 ** -23 * np.abs(y)
    return h, y, dh, dy


def linear(x, dx, qweight, qzeros, scales, group, offset, u=0.0):
    """x [n, K] times a 4-bit linear and the error of an evaluation in fp32 of x known to dx, whose products
    may carry codes and zeros larger by `offset`."""
    K, N = qweight.shape[0], scales.shape[1]
    w, size = np.zeros((K, N)), np.zeros((K, N))
    for i, column in enumerate(ORDER):
        c = ((qweight >> (4 * i)) & 15).astype(np.float64)
        z = np.repeat(((qzeros >> (4 * i)) & 15).astype(np.float64), group, axis=0)
        s = np.repeat(np.asarray(scales, np.float64)[:, column::8], group, axis=0)
        w[:, column::8], size[:, column::8] = (c - z) * s, (c + z + 2 * offset) * np.abs(s)
    steps = 2.0 ** -23 * (group / 16 + K / group + 24)
    return x @ w, steps * (np.abs(x) @ size) + (dx + u * np.abs(x)) @ np.abs(w)


def moe_layer(x, weights, experts, up, down, group, base=None, u=0.0, offset=0):
    """(out, bound of the error before the result's rounding); u: the rounding of the inner activations."""
    T, k = experts.shape
    E, I = up[2].shape[0], up[2].shape[2] // 2
    out = np.zeros((T, down[2].shape[2])) if base is None else np.asarray(base, np.float64).copy()
    bound = 2.0 ** -22 * np.abs(out)
    for t in range(T):
        for j in range(k):
            e = int(experts[t, j])
            if not 0 <= e < E:
                continue
            row = np.asarray(x[t], np.float64)[None]
            both, d = linear(row, np.zeros_like(row), *(a[e] for a in up), group, offset)
            g, v, dg, dv = both[:, :I], both[:, I:], d[:, :I], d[:, I:]
            silu = g / (1 + np.exp(-np.maximum(g, -700.0)))
            act = silu * v
            dact = 1.1 * np.abs(v) * dg + np.abs(silu) * dv + 1.1 * dg * dv + 2.0 ** -20 * np.abs(act)
            y, dy = linear(act, dact, *(a[e] for a in down), group, offset, u)
            w = float(weights[t, j])
            out[t] += w * y[0]
            bound[t] += abs(w) * dy[0] + 2.0 ** -21 * (abs(w) * np.abs(y[0]) + np.abs(out[t]))
    return out, bound

