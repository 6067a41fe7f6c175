"""The attention block of examples/adapted_attention.py with norms of queries and
keys and the 4-bit cache, against the same block in float64.

The reference takes the keys and values as the cache gives them back.  What it
gives back is compared with the exact ones by half a step of the cache (a 15th of
twice the largest magnitude, at most), and 2^-5 of the largest for the roundings
before it: of the projection (2^-8), which the norm's root may add once more,
of the norm's output (2^-8), and of scale and least value (2^-11 each).
The rest: the score's error is a sum over the head of independent roundings of q,
each at most 2 x 2^-8 of a product; 2^-6 of the score's scale, 1, is far beyond it, and
changes each probability by as much, the output by at most twice that.  The
attention's and the last projection's roundings are 2^-8 each: 2^-4 covers all."""

import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def adapted(layer, p, slot, x):
    y = x @ layer.W[p].double().t()
    if slot >= 0:
        A, B, scale = layer.adapters[p, slot]
        y = y + scale * (x @ A.double().t()) @ B.double().t()
    return y


def normed(x, weight):
    return x / ((x * x).mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()


def rotated(x, cos, sin):
    half = x.shape[-1] // 2
    c, s = cos[:x.shape[0], None].double(), sin[:x.shape[0], None].double()
    return torch.cat((x[..., :half] * c - x[..., half:] * s, x[..., half:] * c + x[..., :half] * s), -1)


@pytest.mark.parametrize("head_dim,page", [(64, 16), (128, 64)])
def test_adapted_attention_block_with_norms(head_dim, page):
    from adapted_attention import AdaptedAttention, serve
    from adapter_gemm_linear_gb300 import device_status
    layer = AdaptedAttention(fmt="uint4", page_tokens=page, head_dim=head_dim, norms=True)
    prompts, steps = [100, 37, 1, 260], 5
    xs, ys, table = serve(layer, prompts, steps)
    assert device_status()[0] == 0
    D, G = layer.head_dim, layer.q_heads // layer.kv_heads
    for s, (x, y) in enumerate(zip(xs, ys)):
        n, slot = x.shape[0], s if s < len(prompts) - 1 else -1
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        offs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        k, v = layer.cache.gather(table[s:s + 1].contiguous(), lens, offs, rows=n, dtype=torch.float32)
        xd = x.double()
        q, exact_k = (rotated(normed(adapted(layer, p, slot, xd).view(n, -1, D), w), layer.cos, layer.sin)
                      for p, w in zip("qk", layer.norms))
        exact_v = adapted(layer, "v", slot, xd).view(n, -1, D)
        for got, want in ((k, exact_k), (v, exact_v)):
            assert float((got.double() - want).abs().max()) <= float(want.abs().amax()) * (1.0 / 15 + 2.0 ** -5)
        kd, vd = (t.double().repeat_interleave(G, 1).transpose(0, 1) for t in (k, v))
        scores = q.transpose(0, 1) @ kd.transpose(1, 2) * D ** -0.5
        scores = scores.masked_fill(torch.triu(torch.ones(n, n, dtype=torch.bool, device="cuda"), 1), float("-inf"))
        o = (scores.softmax(-1) @ vd).transpose(0, 1).reshape(n, -1)
        want = adapted(layer, "o", slot, o)
        err = (y.double() - want).abs().amax(1) / want.abs().amax(1)
        assert float(err.max()) <= 2.0 ** -4, f"request {s}: {float(err.max()):.4f}"
