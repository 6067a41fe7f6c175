"""Layouts and ways of calling that include/lora_attention.h promises: heads and rows with gaps between them, outputs that are
part of a larger tensor, tensors with the heads outermost, in place, repeated, and in a graph.

What is compared is the same call on contiguous tensors, bit for bit (a layout changes no arithmetic); the inverse of the
rotary positions is compared with its formula in float64, at test_gpu_attention.py's tolerance."""

import numpy as np
import pytest
import torch

import attention_reference as R
from adapter_gemm_linear_gb300 import KvCache, rope, rope_tables
from test_gpu_attention import DT, FORMATS, dev, draw, setup, status

pytestmark = pytest.mark.gpu

DEV = "cuda"
LAYOUTS = ["heads apart", "columns of a wider row", "heads outermost", "odd pieces"]


def laid_out(x, layout, fill=7.0):
    """(a view with x's values, the tensor behind it, a mask of what lies outside the view)"""
    rows, heads, D = x.shape
    gap = 16 // x.element_size()
    if layout == "heads apart":
        whole = torch.full((rows, heads, D + gap), fill, dtype=x.dtype, device=DEV)
        view = whole[..., :D]
    elif layout == "columns of a wider row":
        whole = torch.full((rows, heads * D + 5 * gap), fill, dtype=x.dtype, device=DEV)
        view = whole[:, gap:gap + heads * D].unflatten(1, (heads, D))  # (16 bytes past a multiple of 32)
    elif layout == "heads outermost":
        whole = torch.full((heads, rows + 1, D), fill, dtype=x.dtype, device=DEV)
        view = whole[:, :rows].transpose(0, 1)
    else:
        whole = torch.full((rows, heads + 1, D + 3 * gap), fill, dtype=x.dtype, device=DEV)
        view = whole[:, 1:, gap:gap + D]
    view.copy_(x)
    inside = torch.zeros_like(whole, dtype=torch.bool)
    inside.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(True)
    return view, whole, ~inside


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,interleaved", [(5, False), (3000, True)])
def test_rope_layouts(layout, dtype, rows, interleaved):
    rng = np.random.default_rng(rows)
    q, k = draw(rng, (rows, 6, 96), dtype)[0].contiguous(), draw(rng, (rows, 2, 96), dtype)[0].contiguous()
    cos, sin = rope_tables(64, 64, device=DEV)
    pos = dev(rng.integers(0, 64, (2, rows)).astype(np.int32))
    args = dict(axes=[i % 2 for i in range(32)], interleaved=interleaved)
    want = rope(q, k, cos, sin, pos, **args)
    ins = [laid_out(t, layout) for t in (q, k)]
    outs = [laid_out(torch.zeros_like(t), layout) for t in (q, k)]
    rope(ins[0][0], ins[1][0], cos, sin, pos, q_out=outs[0][0], k_out=outs[1][0], **args)
    for (view, whole, outside), w in zip(outs, want):
        assert torch.equal(view, w) and bool((whole[outside] == 7).all())
    # in place, q and k both
    rope(ins[0][0], ins[1][0], cos, sin, pos, q_out=ins[0][0], k_out=ins[1][0], **args)
    for (view, whole, outside), w in zip(ins, want):
        assert torch.equal(view, w) and bool((whole[outside] == 7).all())
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,hq,hk,D,rot,axes,interleaved", [
    (7, 5, 3, 128, 128, 1, True), (33, 8, 2, 128, 64, 3, False), (17, 3, 2, 72, 48, 3, True), (2500, 20, 4, 64, 64, 2, True),
])
def test_rope_inverse_forms(dtype, rows, hq, hk, D, rot, axes, interleaved):
    rng = np.random.default_rng(rows + rot)
    q, qd = draw(rng, (rows, hq, D), dtype, pad=16)
    k, kd = draw(rng, (rows, hk, D), dtype)
    cos, sin = rope_tables(300, rot, device=DEV)
    pos = rng.integers(0, 300, (axes, rows)).astype(np.int32)
    ax = rng.integers(0, axes, rot // 2)
    got = rope(q, k, cos, sin, dev(pos), axes=[int(a) for a in ax], interleaved=interleaved, inverse=True)
    c, s = cos.cpu().double().numpy(), sin.cpu().double().numpy()
    for y, x in zip(got, (qd, kd)):
        ref = R.rope(x, c, s, pos, ax, interleaved, inverse=True)
        mag = R.rope(np.abs(x), np.abs(c), np.abs(s), pos, ax, interleaved)
        tol = 2.0 ** -22 * (np.abs(mag) + np.abs(x).max()) + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0)
        assert np.all(np.abs(y.double().cpu().numpy() - ref) <= tol)
    assert status() == 0


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype,D,page", [("bf16", 128, 16), ("fp32", 64, 32), ("bf16", 64, 128), ("fp32", 128, 64)])
def test_cache_layouts(layout, fmt, dtype, D, page):
    news, befores = [3, 1, 40, 0, 130], [10, 127, 0, 5, 14]
    rng, a, table, lens, offs = setup(page + D, news, befores, page, fmt, 3, D)
    b = KvCache(a.num_pages, 3, D, page, fmt)
    for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
        getattr(b, name).copy_(getattr(a, name))
    T = int(offs[-1])
    k, v = draw(rng, (T, 3, D), dtype, 2.0)[0].contiguous(), draw(rng, (T, 3, D), dtype)[0].contiguous()
    args = dev(table), dev(lens), dev(offs)
    a.append(k, v, *args)
    other = LAYOUTS[(LAYOUTS.index(layout) + 1) % len(LAYOUTS)]  # k and v need not be laid out alike
    b.append(laid_out(k, layout)[0], laid_out(v, other)[0], *args)
    for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
        assert torch.equal(getattr(a, name).view(torch.uint8), getattr(b, name).view(torch.uint8)), name
    want = a.gather(*args, rows=T, dtype=DT[dtype])
    outs = laid_out(torch.zeros_like(k), layout), laid_out(torch.zeros_like(v), other)
    a.gather(*args, k_out=outs[0][0], v_out=outs[1][0])
    for (view, whole, outside), w in zip(outs, want):
        assert torch.equal(view, w) and bool((whole[outside] == 7).all())
    assert status() == 0


# (few queries; many, in items that stay whole and in split ones; fp32)
CALLS = [("bf16", [1] * 5, [100, 0, 3000, 17, 700], 128, 16), ("bf16", [1, 4, 2], [9000, 60, 5], 64, 64),
         ("bf16", [40, 90, 7], [0, 33, 500], 128, 16), ("bf16", [300], [7000], 64, 32), ("fp32", [5, 1], [400, 90], 128, 16)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype,news,befores,D,page", CALLS)
def test_attention_layouts(layout, fmt, dtype, news, befores, D, page):
    rng, cache, table, lens, offs = setup(len(news) + D, news, befores, page, fmt, 2, D)
    q = draw(rng, (int(offs[-1]), 10, D), dtype)[0].contiguous()
    args = dev(table), dev(lens), dev(offs)
    want, lse = cache.attention(q, *args, max_queries=max(news), return_lse=True)
    other = LAYOUTS[(LAYOUTS.index(layout) + 1) % len(LAYOUTS)]
    view, whole, outside = laid_out(torch.zeros_like(q), other)
    got, lse2 = cache.attention(laid_out(q, layout)[0], *args, max_queries=max(news), out=view, return_lse=True)
    assert torch.equal(got, want) and torch.equal(lse2, lse) and bool((whole[outside] == 7).all())
    assert status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype,news,befores,D,page", CALLS)
def test_attention_repeats_itself_and_runs_in_a_graph(fmt, dtype, news, befores, D, page):
    """The same bits every time, from a graph too, with the lengths that lie in the tensors when it is replayed."""
    rng, cache, table, lens, offs = setup(3 * len(news) + D, news, befores, page, fmt, 2, D)
    q = draw(rng, (int(offs[-1]), 10, D), dtype)[0].contiguous()
    tb, ln, of = dev(table), dev(lens), dev(offs)

    def call():
        return cache.attention(q, tb, ln, of, max_queries=max(news), return_lse=True)

    want = call()
    for _ in range(5):
        again = call()
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    shorter = dev(np.maximum(lens - 3, np.diff(offs)).astype(np.int32))
    want_shorter = cache.attention(q, tb, shorter, of, max_queries=max(news), return_lse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        captured = call()
    for lengths, w in ((ln.clone(), want), (shorter, want_shorter), (ln.clone(), want)):
        ln.copy_(lengths)
        for t in captured:
            t.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured[0], w[0]) and torch.equal(captured[1], w[1])
    assert status() == 0
