"""Plain numpy restatements, in 64 bits, of the operators between a decoder layer's linears: rotary
positions, attention over a paged cache with a shared prefix, expert routing, dispatch and combine.
Written from the formulas; shares no code with the library."""
from __future__ import annotations

import math

import numpy as np


def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0, beta_fast=32.0, beta_slow=1.0,
                     low_factor=1.0, high_factor=4.0):
    """Angle per position of each of the rot / 2 pairs."""
    out = []
    for i in range(rot // 2):
        if scaling == "ntk":
            stretched = base * factor ** (rot / (rot - 2))
            out.append(stretched ** (-2 * i / rot))
            continue
        f = base ** (-2 * i / rot)
        slow = f / factor
        if scaling == "linear":
            f = slow
        elif scaling == "yarn":
            # the (real) pair index whose frequency turns `beta` times within `original` positions
            index = lambda beta: math.log(original / (2 * math.pi * beta)) / math.log(base) * rot / 2  # noqa: E731
            low, high = max(math.floor(index(beta_fast)), 0), min(math.ceil(index(beta_slow)), rot - 1)
            share = (i - low) / max(high - low, 0.001)
            share = min(max(share, 0.0), 1.0)
            f = share * slow + (1 - share) * f
        elif scaling == "banded":
            wavelength = 2 * math.pi / f
            if wavelength > original / low_factor:
                f = slow
            elif wavelength >= original / high_factor:
                b = (original / wavelength - low_factor) / (high_factor - low_factor)
                f = (1 - b) * slow + b * f
        out.append(f)
    return np.array(out, dtype=np.float64)


def rope(x, positions, frequencies, attention_factor=1.0, interleaved=False):
    """x [T, H, D] rotated, pair by pair, as a product of complex numbers."""
    y = np.array(x, dtype=np.float64)
    half = len(frequencies)
    for i, f in enumerate(frequencies):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        turn = attention_factor * np.exp(1j * np.asarray(positions, dtype=np.float64) * f)[:, None]
        z = (y[:, :, a] + 1j * y[:, :, b]) * turn
        y[:, :, a], y[:, :, b] = z.real, z.imag
    return y


def attention_shared(q, k_cache, v_cache, prefix_pages, prefix_len, pages, lens, scale):
    """q [B, n, Hq, D], caches [pages, page_size, heads, D].  Returns (out, sum_j p_j |v_j|, largest
    scale * sum_d |q_d k_d|): the second and third bound the rounding errors of an implementation."""
    B, n, Hq, D = q.shape
    page, heads = k_cache.shape[1:3]
    group = Hq // heads
    out, spread, largest = np.zeros(q.shape), np.zeros(q.shape), 0.0

    def cells(cache, table, count):
        return np.array([cache[table[j // page], j % page] for j in range(count)], dtype=np.float64).reshape(count, heads, D)

    pk, pv = cells(k_cache, prefix_pages, prefix_len), cells(v_cache, prefix_pages, prefix_len)
    for b in range(B):
        ok, ov = cells(k_cache, pages[b], lens[b]), cells(v_cache, pages[b], lens[b])
        for i in range(n):
            seen = max(0, lens[b] - n + i + 1)
            k, v = np.concatenate([pk, ok[:seen]]), np.concatenate([pv, ov[:seen]])
            if k.shape[0] == 0:
                continue
            for h in range(Hq):
                qh, kh, vh = q[b, i, h].astype(np.float64), k[:, h // group], v[:, h // group]
                z = scale * (kh @ qh)
                largest = max(largest, float(np.max(scale * (np.abs(kh) @ np.abs(qh)))))
                p = np.exp(z - z.max())
                p /= p.sum()
                out[b, i, h], spread[b, i, h] = p @ vh, p @ np.abs(vh)
    return out, spread, largest


def moe_route(logits, k, scoring="softmax", bias=None, groups=1, topk_groups=1, group_best=1, renormalize=True, scale=1.0):
    """Returns (weights [T, k], experts [T, k], clear [T]): clear is False for a row whose choice
    hangs on a difference of under 1e-5 of a key (32-bit scores may order it either way)."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    weights, experts, clear = np.zeros((T, k)), np.full((T, k), -1, dtype=np.int32), np.ones(T, dtype=bool)

    def ranked(values, t, count):
        """The `count` best, best first; only the gaps that decide them count as unclear."""
        order = sorted(range(len(values)), key=lambda e: (-values[e], e))
        for a, b in zip(order[:count], order[1:]):
            gap = values[a] - values[b]
            if 0 < gap < 1e-5 * max(abs(values[a]), 1e-30):
                clear[t] = False
        return order[:count]

    for t in range(T):
        x = logits[t]
        alive = [e for e in range(E) if x[e] != -np.inf]
        if scoring == "sigmoid":
            score = {e: 1 / (1 + math.exp(-x[e])) if x[e] > -700 else 0.0 for e in alive}
        elif alive:
            top = max(x[e] for e in alive)
            mass = {e: math.exp(x[e] - top) for e in alive}
            total = sum(mass.values())
            score = {e: mass[e] / total for e in alive}
        key = {e: score[e] + (0.0 if bias is None else float(bias[e])) for e in alive}
        if groups > 1:
            per, best = E // groups, {}
            for g in range(groups):
                members = sorted((key[e] for e in alive if e // per == g), reverse=True)
                if members:
                    best[g] = sum(members[:group_best])
            names = sorted(best)
            kept = {names[i] for i in ranked([best[g] for g in names], t, topk_groups)}
            alive = [e for e in alive if e // per in kept]
        for j, i in enumerate(ranked([key[e] for e in alive], t, k)):
            experts[t, j], weights[t, j] = alive[i], score[alive[i]]
        total = weights[t].sum()
        if renormalize:
            weights[t] = weights[t] / total if total > 0 else 0.0
        weights[t] *= scale
    return weights, experts, clear


def moe_dispatch(x, experts, E):
    """(routed, offsets, rows) by walking the places expert by expert."""
    T, k = experts.shape
    routed, rows, offsets, done = np.zeros((T * k, x.shape[1]), dtype=x.dtype), np.full((T, k), -1, dtype=np.int32), [0], 0
    for e in range(E):
        for t, j in np.argwhere(experts == e):
            routed[done], rows[t, j] = x[t], done
            done += 1
        offsets.append(done)
    return routed, np.array(offsets, dtype=np.int32), rows


def moe_combine(y, weights, rows, base=None):
    """(out, sum of the magnitudes added)."""
    T, k = rows.shape
    out = np.zeros((T, y.shape[1])) if base is None else base.astype(np.float64)
    size = np.abs(out)
    for t in range(T):
        for j in range(k):
            if 0 <= rows[t, j] < y.shape[0]:
                term = float(weights[t, j]) * y[rows[t, j]].astype(np.float64)
                out[t] += term
                size[t] += np.abs(term)
    return out, size
