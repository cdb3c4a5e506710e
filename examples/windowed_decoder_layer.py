"""Decode steps of a mixture-of-experts decoder layer with 4-bit AWQ weights over a 4-bit key/value cache,
with a sliding window and first tokens that stay visible.  Everything but the router's product runs in the
library, in ten calls:

    q, k, v = qkv(h)                                             AwqLinear
    q rotated; k rotated and v, quantized, into the paged cache   awq_rope_append_kv4
    a   = attention over the window and the first tokens         awq_attention_kv4
    o(a)                                                         AwqLinear
    x   = x + o(a),  h = rms(x)                                  awq_residual_norm
    weights, experts = router logits -> top k                    awq_moe_route
    y   = the routed experts' sum                                awq_moe_layer
    x   = x + scale * rms(y),  h = rms(x) for the next layer     awq_residual_norm

    python examples/windowed_decoder_layer.py        # builds random weights, runs a few steps
"""
import argparse
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import synth  # noqa: E402
import w4a16_weight_only_gb300 as awq  # noqa: E402


def _linear(seed, K, N):
    """Random 4-bit weights of a [K, N] linear whose output keeps its input's size."""
    d = synth.awq_linear(seed, 1, K, N, group_size=128, bias=False)
    scales = (d["scales"].astype(np.float32) * (25.0 / math.sqrt(K))).astype(np.float16)
    return [torch.from_numpy(t).cuda() for t in (d["qweight"], d["qzeros"], scales)]


class Layer:
    """The weights of one layer, its paged 4-bit cache, and the step that runs it."""

    def __init__(self, hidden=1024, heads=16, kv_heads=2, head_dim=64, experts=8, topk=2, ffn=512, page_size=16, pages=256,
                 max_position=4096, window=256, sinks=4, kv_group=64, scale=0.5, seed=0):
        self.heads, self.kv_heads, self.head_dim, self.topk, self.page_size = heads, kv_heads, head_dim, topk, page_size
        self.window, self.sinks, self.kv_group, self.scale = window, sinks, kv_group, scale
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.qkv_weights = _linear(seed + 1, hidden, (heads + 2 * kv_heads) * head_dim)
        self.o_weights = _linear(seed + 2, heads * head_dim, hidden)
        self.qkv, self.o = awq.AwqLinear(*self.qkv_weights), awq.AwqLinear(*self.o_weights)
        up = [_linear(seed + 10 + 2 * e, hidden, 2 * ffn) for e in range(experts)]  # gate and up side by side
        down = [_linear(seed + 11 + 2 * e, ffn, hidden) for e in range(experts)]
        self.up, self.down = ([torch.stack(t) for t in zip(*w)] for w in (up, down))
        self.router = (torch.randn((hidden, experts), generator=g, device="cuda") / math.sqrt(hidden)).half()
        draw = lambda: (1 + 0.1 * torch.randn((hidden,), generator=g, device="cuda")).half()  # noqa: E731
        self.before_experts, self.after_experts, self.next_norm = draw(), draw(), draw()
        self.table = awq.awq_rope_table(max_position, head_dim)
        self.cache = torch.zeros((pages, kv_heads, awq.awq_kv4_page_bytes(page_size, head_dim, kv_group)), dtype=torch.uint8,
                                 device="cuda")

    def project(self, h, positions, slots):
        """Queries [T, heads, head_dim]; the tokens' keys and values go to the cache."""
        T, H, D = h.shape[0], self.heads, self.head_dim
        qkv = self.qkv(h)
        k, v = qkv[:, H * D:].view(T, 2, self.kv_heads, D).unbind(1)
        return awq.awq_rope_append_kv4(qkv[:, :H * D].view(T, H, D), k, v, positions, self.table, self.cache, slots,
                                       group_size=self.kv_group)

    def step(self, x, h, positions, slots, pages, lens):
        """One new token per sequence (at most 16): residual x and normed input h [B, hidden], positions, the
        tokens' cells slots and the lengths with them [B], pages [B, W].  Returns the next layer's x and h."""
        q = self.project(h, positions, slots)
        a = awq.awq_attention_kv4(q, self.cache, pages, lens, group_size=self.kv_group, window=self.window, sinks=self.sinks)
        x, h = awq.awq_residual_norm(self.o(a.flatten(1)), x, weight=self.before_experts)
        weights, experts = awq.awq_moe_route(h @ self.router, self.topk)
        y = awq.awq_moe_layer(h, weights, experts, self.up, self.down)
        return awq.awq_residual_norm(y, x, weight=self.next_norm, post_weight=self.after_experts, scale=self.scale)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=400)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    layer = Layer()
    page, g = layer.page_size, torch.Generator(device="cuda").manual_seed(7)
    per = -(-(a.prompt + a.steps) // page)
    if a.batch * per > layer.cache.shape[0]:
        raise SystemExit(f"the cache has {layer.cache.shape[0]} pages, {a.batch * per} are needed")
    pages = torch.randperm(layer.cache.shape[0], generator=g, device="cuda", dtype=torch.int32)[:a.batch * per].view(a.batch, per)
    at = torch.arange(a.prompt, device="cuda", dtype=torch.int32)
    for b in range(a.batch):  # the prompts' keys and values
        layer.project(torch.randn((a.prompt, 1024), generator=g, device="cuda").half(), at, pages[b, at // page] * page + at % page)
    x = torch.randn((a.batch, 1024), generator=g, device="cuda").half()
    h = x
    for i in range(a.prompt, a.prompt + a.steps):
        position = torch.full((a.batch,), i, dtype=torch.int32, device="cuda")
        x, h = layer.step(x, h, position, (pages[:, i // page] * page + i % page).contiguous(), pages, position + 1)
        print(f"position {i}: residual of {tuple(x.shape)}, rms {x.float().square().mean().sqrt().item():.3f}")
    awq.device_status()


if __name__ == "__main__":
    main()
