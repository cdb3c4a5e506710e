"""The 64-bit oracle of the operators between a layer's linears, pinned on cases worked by hand."""
import math

import numpy as np
import pytest

from oracle import layer


def test_rope_quarter_turn_and_layouts():
    # one pair whose angle is pi / 2 at position 1: (a, b) -> (-b, a)
    x = np.array([[[1.0, 2.0, 7.0]], [[1.0, 2.0, 7.0]]])
    y = layer.rope(x, [0, 1], np.array([math.pi / 2]))
    assert np.allclose(y, [[[1, 2, 7]], [[-2, 1, 7]]])
    x = np.arange(4.0).reshape(1, 1, 4)
    f = np.array([math.pi / 2, math.pi])
    assert np.allclose(layer.rope(x, [1], f), [[[-2, -1, 0, -3]]])                     # pairs (0, 2), (1, 3)
    assert np.allclose(layer.rope(x, [1], f, interleaved=True), [[[-1, 0, -2, -3]]])   # pairs (0, 1), (2, 3)


def test_rope_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(0)
    f = layer.rope_frequencies(16)
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    dot = lambda a, b: float((layer.rope(q, [a], f) * layer.rope(k, [b], f)).sum())  # noqa: E731
    assert dot(3, 9) == pytest.approx(dot(103, 109))
    assert np.linalg.norm(layer.rope(q, [77], f)) == pytest.approx(np.linalg.norm(q))


def test_rope_frequencies():
    f = layer.rope_frequencies(8, base=16.0)
    assert np.allclose(f, [1, 1 / 2, 1 / 4, 1 / 8])
    assert np.allclose(layer.rope_frequencies(8, base=16.0, scaling="linear", factor=4.0), f / 4)
    ntk = layer.rope_frequencies(8, base=16.0, scaling="ntk", factor=8.0)
    assert ntk[0] == 1 and ntk[-1] == pytest.approx(f[-1] / 8)  # the slowest pair is stretched by the factor
    banded = layer.rope_frequencies(8, base=16.0, scaling="banded", factor=2.0, original=2 * math.pi * 8, low_factor=1.5,
                                    high_factor=6.0)
    # turns 8, 4, 2, 1: kept, blended, blended, divided
    assert np.allclose(banded, [1, 0.5 * (1 - 2 / 4.5 / 2), 0.25 * (0.5 + 0.5 * 0.5 / 4.5), 1 / 16])
    yarn = layer.rope_frequencies(8, base=16.0, scaling="yarn", factor=2.0, original=2 * math.pi * 8, beta_fast=8.0, beta_slow=1.0)
    # pair 0 turns 8 times, pair 3 once: a ramp over 0..3
    assert np.allclose(yarn, f * (1 - np.arange(4) / 3 / 2))


def test_attention_counts_keys_once():
    # equal keys: the result is the mean of the values seen
    cache_k, cache_v = np.zeros((3, 2, 1, 4)), np.arange(24.0).reshape(3, 2, 1, 4)
    q = np.ones((1, 2, 2, 4))
    out, _, _ = layer.attention_shared(q, cache_k, cache_v, [2], 1, [[0, 1]], [3], 1.0)
    assert np.allclose(out[0, 0, 0], (cache_v[2, 0, 0] + cache_v[0, 0, 0] + cache_v[0, 1, 0]) / 3)
    assert np.allclose(out[0, 1, 1], (cache_v[2, 0, 0] + cache_v[0, 0, 0] + cache_v[0, 1, 0] + cache_v[1, 0, 0]) / 4)
    out, _, _ = layer.attention_shared(q, cache_k, cache_v, [2], 0, [[0, 1]], [1], 1.0)
    assert np.all(out[0, 0] == 0) and np.allclose(out[0, 1, 0], cache_v[0, 0, 0])  # token 0 sees no key


def test_route_groups_bias_ties():
    x = np.array([[0.0, 1.0, 1.0, -np.inf]])
    w, e, _ = layer.moe_route(x, 3)
    assert e.tolist() == [[1, 2, 0]] and w[0].sum() == pytest.approx(1)
    w, e, _ = layer.moe_route(x, 4)
    assert e.tolist() == [[1, 2, 0, -1]] and w[0, 3] == 0
    x = np.array([[3.0, -3.0, 1.0, 2.0]])
    assert layer.moe_route(x, 2, groups=2, topk_groups=1)[1].tolist() == [[0, 1]]
    assert layer.moe_route(x, 2, scoring="sigmoid", groups=2, topk_groups=1, group_best=2)[1].tolist() == [[3, 2]]
    w, e, _ = layer.moe_route(x, 1, scoring="sigmoid", bias=[0, 1, 0, 0], renormalize=False)
    assert e.tolist() == [[1]] and w[0, 0] == pytest.approx(1 / (1 + math.exp(3)))  # chosen by its bias, weighed without
    assert layer.moe_route(np.full((1, 3), -np.inf), 2)[1].tolist() == [[-1, -1]]


def test_dispatch_then_combine():
    x = np.arange(6, dtype=np.float16).reshape(3, 2)
    experts = np.array([[1, 0], [-1, 1], [1, 5]], dtype=np.int32)
    routed, offsets, rows = layer.moe_dispatch(x, experts, 3)
    assert offsets.tolist() == [0, 1, 4, 4] and rows.tolist() == [[1, 0], [-1, 2], [3, -1]]
    assert routed[:4].tolist() == [[0, 1], [0, 1], [2, 3], [4, 5]] and not routed[4:].any()
    out, _ = layer.moe_combine(routed, np.full((3, 2), 0.5), rows, base=np.ones((3, 2)))
    assert out.tolist() == [[1, 2], [2, 2.5], [3, 3.5]]
