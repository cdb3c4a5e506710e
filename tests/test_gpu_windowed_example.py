"""examples/windowed_decoder_layer.py: decode steps through the 4-bit cache's operators, the norms and the layer
of experts together, against the same steps in 64 bits.

Keys and values are taken from the cache as the step left them (their quantization has bit-exact tests of its
own).  The tensors between the operators are fp16, so a step rounds some 15 times to 2^-11 relative; the norms
keep values near 1 and the sums of a linear average the roundings of its inputs: 1e-2 * max(1, |y|), the
linears' own criterion, leaves room for five roundings in a row at their worst.  Tokens whose experts hang on
a difference of the router's scores below 1e-2 are left out."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from oracle import layer as plain
from oracle import step as plain_step

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from w4a16_weight_only_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("windowed_decoder_layer", os.path.join(ROOT, "examples", "windowed_decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.detach().cpu().double().numpy()


def weights(w):
    return oracle.dequant_f32(*(t.cpu().numpy() for t in w), 128).astype(np.float64)


def norm(x):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)


@pytest.mark.parametrize("B,prompt,window,sinks", [(3, 70, 32, 4), (9, 20, 0, 0)])
def test_steps(example, B, prompt, window, sinks):
    awq = example.awq
    layer = example.Layer(hidden=256, heads=4, kv_heads=2, head_dim=64, experts=4, topk=2, ffn=128, pages=64, window=window,
                          sinks=sinks, kv_group=32, seed=3)
    page, g = layer.page_size, torch.Generator(device="cuda").manual_seed(B)
    layer.cache.fill_(255)
    per = -(-(prompt + 2) // page)
    pages = torch.randperm(64, generator=g, device="cuda", dtype=torch.int32)[:B * per].view(B, per)
    at = torch.arange(prompt, device="cuda", dtype=torch.int32)
    for b in range(B):
        layer.project(torch.randn((prompt, 256), generator=g, device="cuda").half(), at, pages[b, at // page] * page + at % page)
    x = torch.randn((B, 256), generator=g, device="cuda").half()
    h = x
    for i in (prompt, prompt + 1):
        position = torch.full((B,), i, dtype=torch.int32, device="cuda")
        x0, h0 = f64(x), f64(h)
        x, h = layer.step(x, h, position, (pages[:, i // page] * page + i % page).contiguous(), pages, position + 1)
        # the same in 64 bits
        q = (h0 @ weights(layer.qkv_weights))[:, :256].reshape(B, 4, 64)
        q = plain.rope(q, [i] * B, plain.rope_frequencies(64))
        slots = pages.repeat_interleave(page, 1)[:, :i + 1] * page + torch.arange(i + 1, device="cuda", dtype=torch.int32) % page
        keys, values = [], []
        for b in range(B):
            for t, to in zip(awq.awq_kv4_read(layer.cache, slots[b].contiguous(), 64, group_size=32), (keys, values)):
                to.append((f64(t), np.abs(f64(t))))
        a = plain_step.attention(q[:, None], keys, values, [i + 1] * B, 0.125, window, sinks)[0].reshape(B, 256)
        x1, h1 = plain_step.residual_norm(a @ weights(layer.o_weights), x0, weight=f64(layer.before_experts))[:2]
        w, e, _ = plain.moe_route(h1 @ f64(layer.router), 2)
        ranked = np.sort(np.exp(h1 @ f64(layer.router)) / np.exp(h1 @ f64(layer.router)).sum(-1, keepdims=True), axis=-1)
        clear = ranked[:, -2] - ranked[:, -3] > 1e-2
        up, down = ([t[n].cpu().numpy() if n < 2 else f64(t[n]) for n in range(3)] for t in (layer.up, layer.down))
        y = plain_step.moe_layer(h1, w, e, up, down, 128)[0]
        x2, h2 = plain_step.residual_norm(y, x1, weight=f64(layer.next_norm), post_weight=f64(layer.after_experts), scale=0.5)[:2]
        assert clear.sum() >= B // 2
        for got, want in ((x, x2), (h, h2)):
            assert (np.abs(f64(got) - want) <= 1e-2 * np.maximum(1, np.abs(want)))[clear].all()
    awq.device_status()


def test_runs(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["windowed_decoder_layer.py", "--batch", "3", "--prompt", "50", "--steps", "2"])
    example.main()
    assert capsys.readouterr().out.count("residual of (3, 1024)") == 2
