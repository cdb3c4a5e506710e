"""One decode step of a mixture-of-experts decoder layer with 4-bit AWQ weights, for a batch of
sequences that share a prefix: every product and everything between them runs in the library.

    h   = rms(x)                                                (PyTorch)
    q, k, v = qkv(h)                                            AwqLinear
    q rotated; k rotated and v into the paged cache             awq_rope_append
    a   = attention over the shared prefix and each sequence's  awq_attention_shared
    x   = x + o(a)                                              AwqLinear
    weights, experts = router logits -> top k                   awq_moe_route
    rows sorted by expert                                       awq_moe_dispatch
    up / gate, silu, down of the experts                        awq_gemm_grouped
    x   = x + sum of the token's experts                        awq_moe_combine

    python examples/moe_decoder_layer.py            # builds random weights, runs a few steps
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
    """The weights of one layer, its paged cache, and the step that runs it."""

    def __init__(self, hidden=1024, heads=16, kv_heads=2, head_dim=64, experts=8, topk=2, ffn=512, page_size=16, pages=256,
                 max_position=4096, seed=0):
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.experts, self.topk, self.ffn, self.page_size = experts, topk, ffn, page_size
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.qkv_weights = _linear(seed + 1, hidden, (heads + 2 * kv_heads) * head_dim)
        self.o_weights = _linear(seed + 2, heads * head_dim, hidden)
        self.qkv, self.o = awq.AwqLinear(*self.qkv_weights), awq.AwqLinear(*self.o_weights)
        # gate and up projections of an expert side by side
        up = [_linear(seed + 10 + 2 * e, hidden, 2 * ffn) for e in range(experts)]
        down = [_linear(seed + 11 + 2 * e, ffn, hidden) for e in range(experts)]
        self.up, self.down = ([torch.stack(t) for t in zip(*w)] for w in (up, down))
        self.router = (torch.randn((hidden, experts), generator=g, device="cuda") / math.sqrt(hidden)).half()
        self.table = awq.awq_rope_table(max_position, head_dim)
        self.k_cache, self.v_cache = (torch.empty((pages, page_size, kv_heads, head_dim), dtype=torch.float16, device="cuda")
                                      for _ in range(2))

    @staticmethod
    def norm(x):
        y = x.float()
        return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).half()

    def project(self, x, positions, slots):
        """Queries [T, heads, head_dim]; the tokens' keys and values go to the cache."""
        T, H, D = x.shape[0], self.heads, self.head_dim
        qkv = self.qkv(self.norm(x))
        q = qkv[:, :H * D].view(T, H, D)
        k, v = qkv[:, H * D:].view(T, 2, self.kv_heads, D).unbind(1)
        return awq.awq_rope_append(q, k, v, positions, self.table, self.k_cache, self.v_cache, slots)

    def experts_of(self, x):
        """x plus its routed experts' outputs."""
        h = self.norm(x)
        weights, experts = awq.awq_moe_route(h @ self.router, self.topk)
        routed, offsets, rows = awq.awq_moe_dispatch(h, experts, self.experts)
        gate, up = awq.awq_gemm_grouped(routed, *self.up, offsets).split(self.ffn, dim=-1)
        y = awq.awq_gemm_grouped((torch.nn.functional.silu(gate.float()) * up).half(), *self.down, offsets)
        return awq.awq_moe_combine(y, weights, rows, base=x)

    def step(self, x, positions, slots, prefix_pages, prefix_len, pages, lens, max_len):
        """One new token per sequence: x [B, hidden] at positions [B], its cell in the cache at slots [B];
        lens [B] counts a sequence's own tokens, the new one among them."""
        q = self.project(x, positions, slots)
        a = awq.awq_attention_shared(q, self.k_cache, self.v_cache, prefix_pages, prefix_len, pages, lens, max_len=max_len)
        x = x + self.o(a.flatten(1))
        return self.experts_of(x)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--prefix", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    layer = Layer()
    page, g = layer.page_size, torch.Generator(device="cuda").manual_seed(7)
    shared, per = -(-a.prefix // page), -(-a.steps // page)
    order = torch.randperm(layer.k_cache.shape[0], generator=g, device="cuda", dtype=torch.int32)
    if shared + a.batch * per > order.numel():
        raise SystemExit(f"the cache has {order.numel()} pages, {shared + a.batch * per} are needed")
    prefix_pages, pages = order[:shared], order[shared:shared + a.batch * per].view(a.batch, per)
    # the prefix, once for the batch
    at = torch.arange(a.prefix, device="cuda", dtype=torch.int32)
    x = torch.randn((a.prefix, 1024), generator=g, device="cuda").half()
    layer.project(x, at, prefix_pages[at // page] * page + at % page)
    x = torch.randn((a.batch, 1024), generator=g, device="cuda").half()
    for i in range(a.steps):
        position = torch.full((a.batch,), a.prefix + i, dtype=torch.int32, device="cuda")
        slots = pages[:, i // page] * page + i % page
        lens = torch.full((a.batch,), i + 1, dtype=torch.int32, device="cuda")
        x = layer.step(x, position, slots.contiguous(), prefix_pages, a.prefix, pages, lens, i + 1)
        print(f"step {i}: hidden state of {tuple(x.shape)}, rms {x.float().square().mean().sqrt().item():.3f}")
    awq.device_status()


if __name__ == "__main__":
    main()
