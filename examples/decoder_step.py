"""One decoder layer served step by step: attention over a paged key-value cache,
then the MoE block.

    python examples/decoder_step.py [--steps N] [--cache bf16]

A batch of requests has its prompts written to the cache in one call, and then
takes one token a step:

    qkv = x Wqkv                              (library matrix product)
    q   = cache.write_rotary(q, k, v)         rotation, quantised cache write
    o   = cache.attend(q)                     paged attention, one token a request
    x   = MoELayer.forward(o Wo, residual=x)  add + RMSNorm, routing, experts

Weights and inputs are random; every step's attention is compared with a dense
evaluation over the keys and values read back from the cache.
"""

import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from expert_layer_ptpc_gb300 import synthetic as syn  # noqa: E402
from expert_layer_ptpc_gb300.attention import (PagedKVCache, Rotary, frequencies,  # noqa: E402
                                               pair_axes)
from expert_layer_ptpc_gb300.layer import MoELayer  # noqa: E402


class DecoderLayer:
    """Projections, rotation, cache and MoE block of one layer."""

    def __init__(self, cfg, q_heads, kv_heads, head_dim, pages, page_size, cache="e4m3", seed=0):
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(rows, cols):
            w = torch.randn((rows, cols), generator=g, device="cuda") / math.sqrt(rows)
            return w.to(torch.bfloat16)

        self.w_qkv = weight(cfg.D, (q_heads + 2 * kv_heads) * head_dim)
        self.w_o = weight(q_heads * head_dim, cfg.D)
        self.w_router = weight(cfg.D, cfg.E)
        self.gamma = torch.ones(cfg.D, dtype=torch.bfloat16, device="cuda")
        half = head_dim // 2
        third = half // 3
        self.rotary = Rotary(frequencies(head_dim, 1e6),
                             pair_axes([half - 2 * third, third, third], woven=True))
        self.cache = PagedKVCache.empty(pages, kv_heads, page_size, head_dim, dtype=cache)
        self.moe = MoELayer.synthetic(cfg, "cuda", seed)

    def heads(self, x):
        """q, k and v of tokens x, as slices of the projection."""
        qkv = (x @ self.w_qkv).unflatten(1, (-1, self.head_dim))
        return qkv.split([self.q_heads, self.kv_heads, self.kv_heads], 1)

    def prompt(self, x, positions, slots):
        """Write the keys and values of prompt tokens x [T, D] to the cache;
        returns their rotated q."""
        return self.cache.write_rotary(self.rotary, positions, *self.heads(x), slots)

    def step(self, x, positions, slots, table, lengths):
        """One new token a request, x [batch, D]. Returns (the layer's output,
        the residual stream, the attention's output and the rotated q)."""
        q = self.cache.write_rotary(self.rotary, positions, *self.heads(x), slots)
        o = self.cache.attend(q, table, lengths)
        y = o.flatten(1) @ self.w_o
        h = (x.float() + y.float()).to(torch.bfloat16).float()   # what the block normalises
        normed = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6)
        logits = (normed @ self.w_router.float()).contiguous()
        residual = torch.empty_like(x)
        out = self.moe.forward(y, logits, residual=x, gamma=self.gamma, residual_out=residual)
        return out, residual, o, q


def dense_attention(layer, q, table, lengths):
    """Attention over the contexts read back from the cache, in fp64."""
    offsets = torch.zeros(len(lengths) + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(lengths, 0)
    ends = offsets.tolist()
    k, v = layer.cache.read(table, offsets, ends[-1])
    group = layer.q_heads // layer.kv_heads
    outs = []
    for b, (s, e) in enumerate(zip(ends, ends[1:])):
        kb = k[s:e].double().repeat_interleave(group, 1)
        vb = v[s:e].double().repeat_interleave(group, 1)
        scores = torch.einsum("hd,nhd->hn", q[b].double(), kb) / math.sqrt(layer.head_dim)
        outs.append(torch.einsum("hn,nhd->hd", torch.softmax(scores, -1), vb))
    return torch.stack(outs)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=200, help="longest prompt")
    ap.add_argument("--cache", choices=("e4m3", "bf16"), default="e4m3")
    a = ap.parse_args(argv)
    page = 16
    cfg = syn.LayerConfig("decoder", a.batch, 1024, 16, 4, 256, False, "normal")
    each = -(-(a.prompt + a.steps) // page)                # pages of a request
    layer = DecoderLayer(cfg, 16, 2, 128, a.batch * each + 1, page, a.cache)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    table = (torch.randperm(a.batch * each, generator=g, device="cuda") + 1).to(torch.int32)
    table = table.view(a.batch, each)                      # page 0 is nobody's

    def slots_of(b, token):
        return table[b, token // page] * page + token % page

    # prompts of several lengths, in one call
    lengths = torch.tensor([1 + (a.prompt - 1) * i // max(1, a.batch - 1) for i in range(a.batch)],
                           device="cuda")
    b = torch.repeat_interleave(torch.arange(a.batch, device="cuda"), lengths)
    token = torch.cat([torch.arange(n, device="cuda") for n in lengths.tolist()])
    x = torch.randn((len(b), cfg.D), generator=g, device="cuda").to(torch.bfloat16)
    positions = token.to(torch.int32).repeat(3, 1)         # text: the axes agree
    layer.prompt(x, positions, slots_of(b, token).to(torch.int32))

    x = torch.randn((a.batch, cfg.D), generator=g, device="cuda").to(torch.bfloat16)
    every = torch.arange(a.batch, device="cuda")
    worst = 0.0
    for step in range(a.steps):
        positions = lengths.to(torch.int32).repeat(3, 1)
        slots = slots_of(every, lengths).to(torch.int32)
        lengths = lengths + 1
        n = lengths.to(torch.int32)
        out, residual, o, q = layer.step(x, positions, slots, table, n)
        want = dense_attention(layer, q, table, n)
        worst = max(worst, float((o.double() - want).norm() / want.norm()))
        assert layer.moe.status() == (0, 0)
        x = (out.float() + residual.float()).to(torch.bfloat16)
    assert bool(torch.isfinite(x.float()).all())
    print(f"{a.steps} steps of {a.batch} requests, {a.cache} cache: attention within {worst:.1e} "
          f"of a dense evaluation")
    return worst


if __name__ == "__main__":
    main()
