"""The attention block of a decoder layer with an adapter per request: adapted
q/k/v projections, rotary positions (with a norm of every query and key head
before them or without), the 8-bit or 4-bit key/value cache, attention over it,
and the adapted o projection, for prompts and then single tokens.

    python examples/adapted_attention.py [--steps 8] [--fmt uint4] [--norms]

Weights and adapters are random; every request uses its own adapter, the last
one none.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from adapter_gemm_linear_gb300 import KvCache, LoraPool, linear_forward, norm_rope, rope, rope_tables  # noqa: E402


class AdaptedAttention:
    """One layer's attention block; the adapters of slot i belong together in all four projections."""

    def __init__(self, hidden=512, q_heads=8, kv_heads=2, head_dim=64, max_slots=4, rank=8, num_pages=64, page_tokens=16,
                 fmt="int8", max_pos=4096, device="cuda", seed=0, norms=False):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(shape, device=device, generator=g) * std).bfloat16()

        self.q_heads, self.kv_heads, self.head_dim, self.device = q_heads, kv_heads, head_dim, device
        widths = {"q": (q_heads * head_dim, hidden), "k": (kv_heads * head_dim, hidden),
                  "v": (kv_heads * head_dim, hidden), "o": (hidden, q_heads * head_dim)}
        self.W = {p: normal(n, k, std=k ** -0.5) for p, (n, k) in widths.items()}
        self.adapters = {}
        self.pools = {}
        for p, (n, k) in widths.items():
            pool = LoraPool(k, n, max_slots, 16, max_slots, device=device)
            for slot in range(max_slots):
                A, B = normal(rank, k, std=0.05), normal(n, rank, std=0.05)
                pool.load(slot, A, B, alpha=2.0 * rank)
                self.adapters[p, slot] = (A, B, 2.0)
            self.pools[p] = pool
        self.norms = [1.0 + normal(head_dim, std=0.1) for _ in "qk"] if norms else None
        # (decoding fills pages token by token: int8 scales grow by doubling)
        self.cache = KvCache(num_pages, kv_heads, head_dim, page_tokens, fmt, device=device, growth="doubling")
        self.cos, self.sin = rope_tables(max_pos, head_dim, device=device)

    def project(self, x, names, row_adapter):
        outs = [torch.empty((x.shape[0], self.W[p].shape[0]), dtype=x.dtype, device=x.device) for p in names]
        linear_forward(x, [(self.W[p], self.pools[p], out) for p, out in zip(names, outs)], row_adapter=row_adapter)
        return outs

    def forward(self, x, positions, row_adapter, block_table, seq_lens, offsets=None, max_queries=1):
        """x [rows, hidden]: the last tokens of sequences that hold seq_lens tokens with them."""
        q, k, v = self.project(x, "qkv", row_adapter)
        q = q.view(-1, self.q_heads, self.head_dim)
        k, v = (t.view(-1, self.kv_heads, self.head_dim) for t in (k, v))
        if self.norms:
            norm_rope(q, k, *self.norms, self.cos, self.sin, positions, q_out=q, k_out=k)
        else:
            rope(q, k, self.cos, self.sin, positions, q_out=q, k_out=k)
        self.cache.append(k, v, block_table, seq_lens, offsets)
        o = self.cache.attention(q, block_table, seq_lens, offsets, max_queries=max_queries)
        return self.project(o.view(x.shape[0], -1), "o", row_adapter)[0]


def serve(layer: AdaptedAttention, prompts, steps, seed=1):
    """Prompts of these lengths, then `steps` single tokens each, of random
    activations -> (x, y) of all tokens, per request, and the block table."""
    dev, P = layer.device, layer.cache.page_tokens
    S, hidden = len(prompts), layer.W["q"].shape[1]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    xs = [torch.randn((n + steps, hidden), device=dev, generator=g).bfloat16() for n in prompts]
    slots = torch.tensor([s if s < S - 1 else -1 for s in range(S)], dtype=torch.int32, device=dev)
    # every request's pages for all that it will hold
    per = [-(-(n + steps) // P) for n in prompts]
    order = torch.randperm(layer.cache.num_pages, device=dev, generator=g).int()
    table = torch.full((S, max(per)), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(per):
        table[s, :n] = order[at:at + n]
        at += n
    lens = torch.tensor(prompts, dtype=torch.int32, device=dev)
    offsets = torch.zeros(S + 1, dtype=torch.int32, device=dev)
    offsets[1:] = lens.cumsum(0)
    ys = layer.forward(torch.cat([x[:n] for x, n in zip(xs, prompts)]),
                       torch.cat([torch.arange(n, dtype=torch.int32, device=dev) for n in prompts]),
                       slots.repeat_interleave(lens), table, lens, offsets, max_queries=max(prompts))
    out = [list(y.split(1)) for y in ys.split(prompts)]
    for i in range(steps):
        lens = lens + 1
        y = layer.forward(torch.stack([x[n + i] for x, n in zip(xs, prompts)]), lens - 1, slots, table, lens)
        for s in range(S):
            out[s].append(y[s:s + 1])
    return xs, [torch.cat(o) for o in out], table


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--fmt", default="int8", choices=["int8", "e4m3", "uint4"], help="of the cache")
    ap.add_argument("--norms", action="store_true", help="norms of queries and keys")
    args = ap.parse_args()
    layer = AdaptedAttention(fmt=args.fmt, norms=args.norms)
    xs, ys, _ = serve(layer, [100, 37, 5, 260], args.steps)
    for s, (x, y) in enumerate(zip(xs, ys)):
        print(f"request {s}: {x.shape[0]} tokens, |y| {float(y.float().abs().mean()):.4f}")


if __name__ == "__main__":
    main()
