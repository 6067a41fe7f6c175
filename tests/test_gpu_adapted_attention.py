"""The attention block of examples/adapted_attention.py (adapted projections,
rotary positions, 8-bit cache, attention) against the same block in float64.

The 8-bit cache is an approximation by design, so the reference takes the keys
and values as the cache gives them back; what it gives back is compared with
the exact keys and values by the cache's own step (half a step of the page's
largest magnitude over 127, doubled for older tokens rescaled on the way).
Bound of the rest: every bf16 rounding on the way (projection, rotation,
attention, projection) is 2^-8 of its value, of which at most four follow each
other; 2^-5 of the row's largest output covers them."""

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


def rotated(x, cos, sin):
    half = x.shape[-1] // 2
    c, s = cos[:x.shape[0], None].double(), sin[:x.shape[0], None].double()
    return torch.cat((x[..., :half] * c - x[..., half:] * s, x[..., half:] * c + x[..., :half] * s), -1)


@pytest.mark.parametrize("fmt,page", [("int8", 16), ("e4m3", 32)])
def test_adapted_attention_block(fmt, page):
    from adapted_attention import AdaptedAttention, serve
    from adapter_gemm_linear_gb300 import device_status
    layer = AdaptedAttention(fmt=fmt, page_tokens=page)
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
        q = rotated(adapted(layer, "q", slot, xd).view(n, -1, D), layer.cos, layer.sin)
        exact_k = rotated(adapted(layer, "k", slot, xd).view(n, -1, D), layer.cos, layer.sin)
        exact_v = adapted(layer, "v", slot, xd).view(n, -1, D)
        for got, want in ((k, exact_k), (v, exact_v)):
            top = want.abs().amax()
            assert float((got.double() - want).abs().max()) <= float(top) * (2.0 / 127 + 2.0 ** -6 if fmt == "int8" else 2.0 ** -3)
        kd, vd = (t.double().repeat_interleave(G, 1).transpose(0, 1) for t in (k, v))
        scores = q.transpose(0, 1) @ kd.transpose(1, 2) * D ** -0.5
        scores = scores.masked_fill(torch.triu(torch.ones(n, n, dtype=torch.bool, device="cuda"), 1), float("-inf"))
        o = (scores.softmax(-1) @ vd).transpose(0, 1).reshape(n, -1)
        want = adapted(layer, "o", slot, o)
        err = (y.double() - want).abs().amax(1) / want.abs().amax(1)
        assert float(err.max()) <= 2.0 ** -5, f"request {s}: {float(err.max()):.4f}"
