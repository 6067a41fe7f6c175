"""GPU parity of lora_norm_rope and its gradient with plain float64 restatements.

Tolerances, u = 2^-24 (half a step of fp32's, relative):
  r = 1 / sqrt(mean(x^2) + eps): a lane's squares are a chain of 16 at most and five
  sums by shuffles, 23 u of the sum with its own rounding, half of that in r; the mean
  and eps 2 u, halved too; rsqrtf two steps, 4 u: below 17 u.
  y: r, two products, a product and a sum of the rotation: below 22 u of |n1| + |n2|, 2^-19.5;
  dx = r (a - x r^2 mean(a x)): with G = (|g1| + |g2|) |W| and A = mean |a x|, the first term
  is off by 4 u (h, times W), the second by 4 + 23 (mean) + 35 (r^2) + 3 u, and both by 18 u
  (r) and the two last roundings: below 2^-17.5 r (G + |x| r^2 A);
  dw: its terms by 22 u each; the longest chain of its sums is what a thread has of rows and
  heads, then the block's groups (128 at most) and the blocks: below 512 in the cases here, so
  below 2^-14.9 of the sum of |h x r|.
bf16 results have one rounding more, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import attention_reference as R
from adapter_gemm_linear_gb300 import LoraError, device_status, norm_rope, norm_rope_backward, rope, rope_tables
from test_gpu_attention import DT, dev, draw, status
from test_gpu_attention_layouts import LAYOUTS, laid_out

pytestmark = pytest.mark.gpu

DEV = "cuda"
EPS = 1e-5
EPS32 = float(np.float32(EPS))


def forward(x, W, cos, sin, pos, ax, interleaved, eps=EPS32):
    """float64 x [rows, heads, D], W [D] -> (n, y)"""
    n = x * W / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return n, R.rope(n, cos, sin, pos, ax, interleaved)


def backward(g, x, W, cos, sin, pos, ax, interleaved, eps=EPS32):
    """-> dx, its tolerance's scale, dw, the sum of |h x r|"""
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = R.rope(g, cos, sin, pos, ax, interleaved, inverse=True)
    a = h * W
    dx = r * (a - x * r * r * (a * x).mean(-1, keepdims=True))
    half = cos.shape[1]
    both = np.abs(g).copy()
    for i in range(half):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        both[..., p] = both[..., q] = np.abs(g[..., p]) + np.abs(g[..., q])
    G = both * np.abs(W)
    scale = r * (G + np.abs(x) * r * r * (G * np.abs(x)).mean(-1, keepdims=True))
    return dx, scale, (h * x * r).sum((0, 1)), (both * np.abs(x) * r).sum((0, 1))


SHAPES = [  # rows, q heads, k heads, D, rot, axes, interleaved
    (1, 1, 1, 64, 64, 1, False), (7, 5, 3, 128, 128, 1, True), (33, 32, 8, 128, 128, 3, False),
    (5, 4, 0, 80, 32, 2, False), (17, 3, 2, 72, 48, 3, True), (900, 40, 8, 128, 128, 3, False),
    (1200, 33, 4, 96, 64, 1, True), (3, 2, 1, 256, 256, 1, False), (260, 16, 1, 256, 64, 2, True),
    (2, 1, 40, 16, 16, 1, False), (6, 100, 30, 248, 16, 1, False), (400, 1, 70, 256, 128, 1, True),
    (3, 2, 300, 64, 64, 1, False),
]


def make(rows, hq, hk, D, rot, axes, dtype, width=3.0, offset=False):
    rng = np.random.default_rng(rows * 7 + D)
    q, qd = draw(rng, (rows, hq, D), dtype, width, pad=16)
    k, kd = draw(rng, (rows, hk, D), dtype, width, pad=8) if hk else (None, None)
    cos, sin = rope_tables(501, rot, device=DEV)
    pos = rng.integers(0, 501, (axes, rows)).astype(np.int32)
    pos[0, 0], pos[-1, -1] = 0, 500
    ax = [int(a) for a in rng.integers(0, axes, rot // 2)]
    w = torch.from_numpy((rng.normal(size=(2, D)) * 0.4 + (0 if offset else 1)).astype(np.float32))
    return rng, q, qd, k, kd, cos, sin, pos, ax, w


@pytest.mark.parametrize("dtype,wtype,offset", [("bf16", "bf16", False), ("fp32", "fp32", True), ("bf16", "fp32", True)])
@pytest.mark.parametrize("rows,hq,hk,D,rot,axes,interleaved", SHAPES)
def test_norm_rope(dtype, wtype, offset, rows, hq, hk, D, rot, axes, interleaved):
    rng, q, qd, k, kd, cos, sin, pos, ax, w = make(rows, hq, hk, D, rot, axes, dtype, offset=offset)
    w = w.to(DT[wtype])
    args = dict(eps=EPS, unit_offset=offset, axes=ax, interleaved=interleaved)
    p = dev(pos) if axes > 1 else dev(pos[0])
    wq, wk = w[0].to(DEV), w[1].to(DEV)
    got = norm_rope(q, k, wq, wk if hk else None, cos, sin, p, **args)
    g, gd = draw(rng, (rows, hq, D), dtype, pad=24)
    gk, gkd = draw(rng, (rows, hk, D), dtype) if hk else (None, None)
    grads = norm_rope_backward(g, gk, q, k, wq, wk if hk else None, cos, sin, p, **args)
    c, s = cos.cpu().double().numpy(), sin.cpu().double().numpy()
    for i, (x, gx) in enumerate(((qd, gd), (kd, gkd))):
        if x is None:
            assert got[i] is None and grads[i] is None and grads[2 + i] is None
            continue
        W = w[i].double().numpy() + offset
        n, ref = forward(x, W, c, s, pos, ax, interleaved)
        mag = R.rope(np.abs(n), np.ones_like(c), -np.ones_like(s), pos, ax, interleaved)  # (|n1| + |n2| in the first of a pair)
        mag = np.maximum(np.abs(mag), np.abs(R.rope(np.abs(n), np.ones_like(c), np.ones_like(s), pos, ax, interleaved)))
        tol = 2.0 ** -19.5 * mag + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0)
        assert got[i].dtype == q.dtype
        assert np.all(np.abs(got[i].double().cpu().numpy() - ref) <= tol)
        dx, scale, dw, total = backward(gx, x, W, c, s, pos, ax, interleaved)
        tol = 2.0 ** -17.5 * scale + (2.0 ** -8 * np.abs(dx) if dtype == "bf16" else 0)
        assert grads[i].dtype == q.dtype and grads[2 + i].dtype == torch.float32
        assert np.all(np.abs(grads[i].double().cpu().numpy() - dx) <= tol)
        assert np.all(np.abs(grads[2 + i].double().cpu().numpy() - dw) <= 2.0 ** -14.9 * total)
    # the same bits again, and in place
    assert all(a is None or torch.equal(a, b) for a, b in
               zip(grads, norm_rope_backward(g, gk, q, k, wq, wk if hk else None, cos, sin, p, **args)))
    q2, g2, g3 = q.clone(), g.clone(), q.clone()
    assert torch.equal(norm_rope(q2, None, wq, None, cos, sin, p, q_out=q2, **args)[0], got[0])
    assert torch.equal(norm_rope_backward(g2, None, q, None, wq, None, cos, sin, p, q_out=g2, **args)[0], grads[0])
    assert torch.equal(norm_rope_backward(g, None, g3, None, wq, None, cos, sin, p, q_out=g3, **args)[0], grads[0])
    assert status() == 0


@pytest.mark.parametrize("dtype,rows,hq,hk,D,rot,axes,interleaved", [
    ("bf16", 8300, 32, 7, 64, 64, 2, False), ("bf16", 8300, 38, 0, 64, 48, 1, True), ("bf16", 4150, 33, 5, 128, 128, 3, False),
    ("bf16", 4150, 11, 28, 128, 128, 1, True), ("bf16", 2100, 31, 8, 256, 256, 1, False), ("bf16", 1300, 25, 8, 248, 16, 1, True),
    ("fp32", 4150, 31, 8, 64, 64, 1, True), ("fp32", 2100, 37, 2, 128, 128, 2, False), ("fp32", 1250, 2, 30, 256, 64, 2, False),
])
def test_many_rows(dtype, rows, hq, hk, D, rot, axes, interleaved):
    """The kernel that takes rows in turns: groups of 4, 8, 16 and 32 lanes, and two chunks a lane."""
    test_norm_rope(dtype, dtype, True, rows, hq, hk, D, rot, axes, interleaved)


def test_gradient_against_differences():
    """The kernel's gradient against central differences of the float64 formula that the forward pass is tested against."""
    rng, q, qd, _, _, cos, sin, pos, ax, w = make(3, 2, 0, 32, 16, 2, "fp32")
    g, gd = draw(rng, (3, 2, 32), "fp32")
    c, s = cos.cpu().double().numpy(), sin.cpu().double().numpy()
    W = w[0].double().numpy()

    def loss(x, W):
        return float((forward(x, W, c, s, pos, ax, True)[1] * gd).sum())

    got = norm_rope_backward(g, None, q, None, w[0].to(DEV), None, cos, sin, dev(pos), eps=EPS, axes=ax, interleaved=True)
    h = 2.0 ** -14
    dx, dw = got[0].double().cpu().numpy(), got[2].double().cpu().numpy()
    for i in rng.integers(0, qd.size, 40):
        e = np.zeros(qd.size)
        e[i] = h
        e = e.reshape(qd.shape)
        want = (loss(qd + e, W) - loss(qd - e, W)) / (2 * h)
        assert abs(dx.flat[i] - want) <= 1e-5  # (h^2 / 6 of a third derivative below 100, and 2^-17.5 of values below 1)
    for d in range(32):
        e = np.zeros(32)
        e[d] = h
        want = (loss(qd, W + e) - loss(qd, W - e)) / (2 * h)  # (linear in W)
        assert abs(dw[d] - want) <= 1e-5 * max(1.0, abs(want))


def test_without_weights_and_with_one():
    rng, q, qd, k, kd, cos, sin, pos, ax, w = make(9, 4, 2, 64, 64, 1, "fp32")
    wk = w[1].to(DEV)
    p = dev(pos[0])
    got = norm_rope(q, k, None, wk, cos, sin, p, eps=EPS)
    ones = torch.ones(64, device=DEV)
    want = norm_rope(q, k, ones, wk, cos, sin, p, eps=EPS)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # unit_offset says nothing about a weight that is not there
    assert torch.equal(norm_rope(q, None, None, None, cos, sin, p, eps=EPS, unit_offset=True)[0], want[0])
    b = norm_rope_backward(q, k, q, k, None, wk, cos, sin, p, eps=EPS)
    c = norm_rope_backward(q, k, q, k, ones, wk, cos, sin, p, eps=EPS)
    assert b[2] is None and torch.equal(b[0], c[0]) and torch.equal(b[1], c[1]) and torch.equal(b[3], c[3])
    n = norm_rope_backward(q, None, q, None, None, None, cos, sin, p, eps=EPS)
    assert n[2] is None and n[3] is None and torch.equal(n[0], c[0])


def test_zeros_infinities_and_nan_stay_in_their_head():
    x = torch.randn((4, 3, 64), device=DEV)
    x[0, 0] = 0
    x[1, 1, 5] = float("inf")
    x[2, 2, 7] = float("nan")
    cos, sin = rope_tables(8, 64, device=DEV)
    p = torch.arange(4, dtype=torch.int32, device=DEV)
    w = torch.ones(64, device=DEV)
    y = norm_rope(x, None, w, None, cos, sin, p)[0]
    clean = x.clone()
    clean[1, 1, 5] = clean[2, 2, 7] = 1.0
    z = norm_rope(clean, None, w, None, cos, sin, p)[0]
    bad = torch.zeros((4, 3), dtype=torch.bool, device=DEV)
    bad[1, 1] = bad[2, 2] = True
    assert torch.equal(y[~bad], z[~bad]) and bool((y[0, 0] == 0).all())
    assert bool(y[1, 1].isnan().any()) and bool(y[2, 2].isnan().all())


def test_positions_out_of_range():
    x = torch.randn((3, 2, 64), device=DEV)
    cos, sin = rope_tables(8, 64, device=DEV)
    status()
    pos = dev(np.array([3, 8, -1], np.int32))
    for interleaved in (False, True):
        y = norm_rope(x, None, None, None, cos, sin, pos, interleaved=interleaved)[0]
        st, row = device_status()
        assert st == 11 and row in (1, 2)
        at0 = norm_rope(x, None, None, None, cos, sin, torch.zeros_like(pos), interleaved=interleaved)[0]  # the angle 0
        assert torch.equal(y[1:], at0[1:]) and not torch.equal(y[0], at0[0])
        g = norm_rope_backward(x, None, x, None, None, None, cos, sin, pos, interleaved=interleaved)[0]
        assert device_status()[0] == 11
        g0 = norm_rope_backward(x, None, x, None, None, None, cos, sin, torch.zeros_like(pos), interleaved=interleaved)[0]
        assert torch.equal(g[1:], g0[1:]) and not torch.equal(g[0], g0[0])
    assert status() == 0


def test_no_rows():
    x = torch.empty((0, 2, 64), device=DEV)
    cos, sin = rope_tables(8, 64, device=DEV)
    p = torch.empty(0, dtype=torch.int32, device=DEV)
    w = torch.ones(64, device=DEV)
    assert norm_rope(x, x, w, w, cos, sin, p)[1].shape == (0, 2, 64)
    g = norm_rope_backward(x, x, x, x, w, w, cos, sin, p)
    assert bool((g[2] == 0).all()) and bool((g[3] == 0).all())


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype,rows", [("bf16", 1500), ("fp32", 5)])
def test_layouts(layout, dtype, rows):
    rng, q, _, k, _, cos, sin, pos, ax, w = make(rows, 6, 2, 96, 64, 2, dtype)
    q, k = q.contiguous(), k.contiguous()
    g, gk = draw(rng, (rows, 6, 96), dtype)[0].contiguous(), draw(rng, (rows, 2, 96), dtype)[0].contiguous()
    w = w.to(DEV)
    args = dict(axes=ax)
    rest = (w[0], w[1], cos, sin, dev(pos))
    want, wantg = norm_rope(q, k, *rest, **args), norm_rope_backward(g, gk, q, k, *rest, **args)
    ins = [laid_out(t, layout)[0] for t in (q, k, g, gk)]
    outs = [laid_out(torch.zeros_like(t), layout) for t in (q, k, q, k)]
    norm_rope(ins[0], ins[1], *rest, q_out=outs[0][0], k_out=outs[1][0], **args)
    got = norm_rope_backward(ins[2], ins[3], ins[0], ins[1], *rest, q_out=outs[2][0], k_out=outs[3][0], **args)
    for (view, whole, outside), x in zip(outs, want + wantg[:2]):
        assert torch.equal(view, x) and bool((whole[outside] == 7).all())
    assert torch.equal(got[2], wantg[2]) and torch.equal(got[3], wantg[3])


def test_streams_and_graphs():
    """On another stream, in two graphs over one workspace, and replayed with new inputs."""
    rng, q, _, k, _, cos, sin, pos, ax, w = make(700, 16, 4, 128, 128, 1, "bf16")
    g, gk = draw(rng, (700, 16, 128), "bf16")[0], draw(rng, (700, 4, 128), "bf16")[0]
    w, p = w.to(DEV), dev(pos[0])
    rest = (w[0], w[1], cos, sin, p)
    want = norm_rope(q, k, *rest) + norm_rope_backward(g, gk, q, k, *rest)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = norm_rope(q, k, *rest, stream=side) + norm_rope_backward(g, gk, q, k, *rest, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    space = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(norm_rope(q, k, *rest) + norm_rope_backward(g, gk, q, k, *rest, workspace=space))
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    q.mul_(-0.5), g.mul_(2.0)
    graphs[0].replay()
    want = norm_rope(q, k, *rest) + norm_rope_backward(g, gk, q, k, *rest)
    assert all(torch.equal(a, b) for a, b in zip(outs[0], want))


def test_binding_refusals():
    x = torch.zeros((2, 2, 64), device=DEV)
    cos, sin = rope_tables(8, 64, device=DEV)
    p = torch.zeros(2, dtype=torch.int32, device=DEV)
    w = torch.ones(64, device=DEV)
    rest = (cos, sin, p)
    for bad in (w[:32], w.bfloat16(), w.cpu(), torch.ones(128, device=DEV)[::2]):
        with pytest.raises(ValueError):
            norm_rope(x, x, w, bad, *rest)
    with pytest.raises(TypeError):
        norm_rope(x, x, w.half(), w.half(), *rest)
    with pytest.raises(LoraError):
        norm_rope(x, x, w, w, *rest, eps=0.0)
    with pytest.raises(LoraError):
        norm_rope(x.repeat(1, 1, 5), None, None, None, *rest)
    with pytest.raises(ValueError):
        norm_rope_backward(x[:1], x, x, x, w, w, *rest)
    with pytest.raises(ValueError):
        norm_rope_backward(x, None, x, x, w, w, *rest)
    with pytest.raises(ValueError):
        norm_rope_backward(x, x.bfloat16(), x, x, w, w, *rest)
    with pytest.raises(LoraError):
        norm_rope_backward(x, x, x, x, w, w, *rest, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    # positions far beyond the heads' number of rows are no matter of the norm: rope's own refusals hold
    with pytest.raises(ValueError):
        norm_rope(x, x, w, w, cos, sin, p[:1])
    assert torch.equal(norm_rope(x, x, w, w, *rest)[0], rope(x, x, *rest)[0])  # zeros
