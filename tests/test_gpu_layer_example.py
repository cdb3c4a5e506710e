"""examples/moe_decoder_layer.py: one decode step through every operator between the linears, against the
same step in 64 bits from the dequantized weights.

The tensors between the operators are fp16, so the step rounds some 15 times to 2^-11 relative; the
norms keep values near 1 and the sums of a linear average the roundings of its inputs.  1e-2 * max(1,
|y|), the linears' own criterion, leaves room for five roundings in a row at their worst.  Tokens whose
experts hang on a difference of the router's scores below 1e-2 are left out."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import oracle
from oracle import layer as plain

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from w4a16_weight_only_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("moe_decoder_layer", os.path.join(ROOT, "examples", "moe_decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.detach().cpu().double().numpy()


def weights(w):
    return oracle.dequant_f32(*(t.cpu().numpy() for t in w), 128).astype(np.float64)


def norm(x):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)


@pytest.mark.parametrize("B,prefix", [(5, 37), (40, 130)])
def test_step(example, B, prefix):
    layer = example.Layer(hidden=256, heads=4, kv_heads=2, head_dim=64, experts=4, topk=2, ffn=128, pages=128, seed=3)
    page, g = layer.page_size, torch.Generator(device="cuda").manual_seed(B)
    layer.k_cache.fill_(float("nan"))
    layer.v_cache.fill_(float("nan"))
    shared = -(-prefix // page)
    order = torch.randperm(128, generator=g, device="cuda", dtype=torch.int32)
    pp, pages = order[:shared], order[shared:shared + B].view(B, 1)
    own = 3  # tokens a sequence has of its own, the new one among them
    at = torch.arange(prefix, device="cuda", dtype=torch.int32)
    xs = [torch.randn((prefix, 256), generator=g, device="cuda").half()]
    layer.project(xs[0], at, pp[at // page] * page + at % page)
    for i in range(own):
        xs.append(torch.randn((B, 256), generator=g, device="cuda").half())
        pos = torch.full((B,), prefix + i, dtype=torch.int32, device="cuda")
        slots = (pages[:, 0] * page + i).contiguous()
        if i + 1 < own:
            layer.project(xs[-1], pos, slots)
    lens = torch.full((B,), own, dtype=torch.int32, device="cuda")
    out = f64(layer.step(xs[-1], pos, slots, pp, prefix, pages, lens, own))

    # the same in 64 bits
    H, KV, D = 4, 2, 64
    wq, wo = weights(layer.qkv_weights), weights(layer.o_weights)
    freq = plain.rope_frequencies(D)

    def project(x, position):
        y = norm(f64(x)) @ wq
        T = y.shape[0]
        q = plain.rope(y[:, :H * D].reshape(T, H, D), position, freq)
        k = plain.rope(y[:, H * D:(H + KV) * D].reshape(T, KV, D), position, freq)
        return q, k, y[:, (H + KV) * D:].reshape(T, KV, D)

    kc, vc = np.zeros((128, page, KV, D)), np.zeros((128, page, KV, D))
    _, k, v = project(xs[0], np.arange(prefix))
    table = pp.tolist()
    for j in range(prefix):
        kc[table[j // page], j % page], vc[table[j // page], j % page] = k[j], v[j]
    for i in range(own):
        q, k, v = project(xs[1 + i], np.full(B, prefix + i))
        for b in range(B):
            kc[pages[b, 0], i], vc[pages[b, 0], i] = k[b], v[b]
    a, _, _ = plain.attention_shared(q[:, None], kc, vc, table, prefix, pages.tolist(), [own] * B, 1 / math.sqrt(D))
    x = f64(xs[-1]) + a.reshape(B, H * D) @ wo
    h = norm(x)
    logits = h @ f64(layer.router)
    w, e, _ = plain.moe_route(logits, 2)
    ranked = np.sort(logits, axis=1)[:, ::-1]
    clear = (ranked[:, :2] - ranked[:, 1:3]).min(1) > 1e-2
    y = x.copy()
    for b in range(B):
        for j in range(2):
            up = h[b] @ weights([t[e[b, j]] for t in layer.up])
            gate, up = up[:128], up[128:]
            y[b] += w[b, j] * ((gate / (1 + np.exp(-gate)) * up) @ weights([t[e[b, j]] for t in layer.down]))
    assert clear.mean() > 0.5
    assert (np.abs(out - y) <= 1e-2 * np.maximum(1, np.abs(y)))[clear].all()


def test_main(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["moe_decoder_layer.py", "--batch", "6", "--prefix", "50", "--steps", "2"])
    example.main()
    assert capsys.readouterr().out.count("rms") == 2
