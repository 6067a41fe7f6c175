"""GPU parity of rotary positions, the 8-bit paged cache and attention over it
(include/lora_attention.h) with plain float64 restatements.

Tolerances, per output value o:
  codes and scales: equal, bit for bit (both sides do the definition's fp32 steps);
  gathered values: one rounding of code * scale: 2^-24 |o| in fp32, 2^-8 |o| in bf16
  (8 significant bits, half of their spacing at worst);
  rope: three fp32 roundings (2^-22 (|x1| + |x2|)), in bf16 one more (2^-8 |o|);
  attention, with A = sum p |v| and S = scale * sum |q k| (the row's largest),
  n keys, V the largest |v|:
    bf16: 2^-8 |o| (its rounding) + A (2^-11 (p's 11 bits) + 2^-20 (S + 16))
          + n 2^-25 V (the least step of p's format)
    fp32: A (2^-21 (22 bits of p) + 2^-20 (S + 16)) + 2^-23 |o| + n 2^-36 V
    lse:  2^-20 (S + 16).
  (scores are fp32 sums of exact products, off by less than 2^-20 S; 16 covers
  the exponential and the fp32 sums.)
"""

import numpy as np
import pytest
import torch

import attention_reference as R
from adapter_gemm_linear_gb300 import KvCache, LoraError, device_status, rope, rope_tables

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
FORMATS = ["int8", "e4m3"]


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def draw(rng, shape, dtype, width=1.0, pad=0):
    """(device tensor of the dtype, its values in float64); pad: extra columns between the rows."""
    x = torch.from_numpy(rng.normal(size=shape[:1] + (shape[1] * shape[2] + pad,)).astype(np.float32) * width).to(DT[dtype])
    t = x.to(DEV)[:, :shape[1] * shape[2]].unflatten(1, shape[1:])
    return t, x[:, :shape[1] * shape[2]].double().numpy().reshape(shape)


def status():
    return device_status()[0]


# ---------------------------------------------------------------- rope

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,hq,hk,D,rot,axes,interleaved", [
    (1, 1, 1, 64, 64, 1, False), (7, 5, 3, 128, 128, 1, True), (33, 32, 8, 128, 128, 3, False),
    (5, 4, 0, 80, 32, 2, False), (17, 3, 2, 72, 48, 3, True), (2500, 40, 8, 128, 128, 3, False),
    (3000, 33, 4, 96, 64, 1, True),
])
def test_rope(dtype, rows, hq, hk, D, rot, axes, interleaved):
    rng = np.random.default_rng(rows * 7 + D)
    q, qd = draw(rng, (rows, hq, D), dtype, pad=16)
    k, kd = draw(rng, (rows, hk, D), dtype, pad=8) if hk else (None, None)
    cos, sin = rope_tables(501, rot, device=DEV)
    pos = rng.integers(0, 501, (axes, rows)).astype(np.int32)
    pos[0, 0], pos[-1, -1] = 0, 500
    ax = rng.integers(0, axes, rot // 2)
    args = dict(axes=[int(a) for a in ax], interleaved=interleaved)
    p = dev(pos) if axes > 1 else dev(pos[0])
    qo, ko = rope(q, k, cos, sin, p, **args)
    assert (ko is None) == (hk == 0)
    c, s = cos.cpu().double().numpy(), sin.cpu().double().numpy()
    for got, x in ((qo, qd), (ko, kd)):
        if got is None:
            continue
        ref = R.rope(x, c, s, pos, ax, interleaved)
        mag = R.rope(np.abs(x), np.abs(c), np.abs(s), pos, ax, interleaved, inverse=False)
        tol = 2.0 ** -22 * (np.abs(mag) + np.abs(x).max()) + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0)
        assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)
    # in place gives the same bits, and dimensions past rot are the input's
    assert torch.equal(qo[..., rot:], q[..., rot:])
    q2 = q.clone()
    rope(q2, None, cos, sin, p, q_out=q2, **args)
    assert torch.equal(q2, qo)
    assert status() == 0


def test_rope_gradient_is_the_inverse():
    rng = np.random.default_rng(5)
    x, xd = draw(rng, (6, 2, 64), "fp32")
    g, gd = draw(rng, (6, 2, 64), "fp32")
    cos, sin = rope_tables(64, 64, device=DEV)
    pos = dev(rng.integers(0, 64, 6).astype(np.int32))
    dx = rope(g, None, cos, sin, pos, inverse=True)[0]
    # against the formula: the gradient of sum(g * rope(x)) by x
    ref = R.rope(gd, cos.cpu().double().numpy(), sin.cpu().double().numpy(), pos.cpu().numpy()[None], [0] * 32, False, True)
    assert np.all(np.abs(dx.double().cpu().numpy() - ref) <= 2.0 ** -21 * np.abs(gd).max())
    # and against differences (rope is linear: any step gives the slope, up to fp32 rounding of the two values)
    u, _ = draw(rng, (6, 2, 64), "fp32")
    slope = (rope(x + u, None, cos, sin, pos)[0].double() * g.double()).sum() - \
        (rope(x - u, None, cos, sin, pos)[0].double() * g.double()).sum()
    want = 2 * (dx.double() * u.double()).sum()
    scale = (g.abs().double() * (x.abs() + u.abs()).double()).sum()
    assert abs(float(slope - want)) <= 2.0 ** -20 * float(scale)
    # and it undoes the call
    y = rope(x, None, cos, sin, pos)[0]
    z = rope(y, None, cos, sin, pos, inverse=True)[0]
    assert float((z - x).abs().max()) <= 2.0 ** -20 * float(x.abs().max())


def test_rope_reports_positions_out_of_range():
    x = torch.randn((3, 1, 64), device=DEV)
    cos, sin = rope_tables(8, 64, device=DEV)
    status()
    y = rope(x, None, cos, sin, dev(np.array([3, 8, -1], np.int32)))[0]
    st, row = device_status()
    assert st == 11 and row in (1, 2)
    assert torch.equal(y[1:], x[1:]) and not torch.equal(y[0], x[0])


# ---------------------------------------------------------------- cache

def check_cache(cache, ref, table, lens, offs, back):
    """Codes of the sequences' last `back[s]` tokens, and all scales, equal the reference's."""
    k, v = R.unpack_k(cache.k_pages), R.unpack_v(cache.v_pages)
    for s in range(len(lens)):
        for j in range(lens[s] - back[s], lens[s]):
            page, t = table[s][j // ref.P], j % ref.P
            np.testing.assert_array_equal(k[page, :, t], ref.k[page, :, t], err_msg=f"k seq {s} token {j}")
            np.testing.assert_array_equal(v[page, :, t], ref.v[page, :, t], err_msg=f"v seq {s} token {j}")
    np.testing.assert_array_equal(cache.k_scales.cpu().numpy(), ref.ks)
    np.testing.assert_array_equal(cache.v_scales.cpu().numpy(), ref.vs)


BATCHES = [
    ([1], [0]), ([1, 1, 1], [0, 15, 16]), ([1] * 6, [3, 127, 64, 31, 0, 200]), ([40], [0]), ([129], [7]),
    ([3, 0, 50, 16, 1], [0, 9, 14, 16, 100]), ([2, 0, 33], [30, 0, 95]),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,D,H", [("bf16", 128, 2), ("fp32", 64, 3), ("bf16", 64, 1), ("fp32", 128, 5)])
def test_append_and_gather(fmt, page, dtype, D, H):
    for i, (news, befores) in enumerate(BATCHES):
        rng = np.random.default_rng(i * 100 + page + D)
        table, lens, offs, num = R.make_batch(rng, news, befores, page)
        cache = KvCache(num, H, D, page, fmt)
        R.random_codes(rng, cache)
        ref = R.Paged(cache)
        T = int(offs[-1])
        k, kd = draw(rng, (T, H, D), dtype, 3.0, pad=8)
        v, vd = draw(rng, (T, H, D), dtype, 0.2, pad=24)
        tb, ln, of = dev(table), dev(lens), dev(offs)
        ones = all(n == 1 for n in news)
        cache.append(k, v, tb, ln, None if ones else of)
        R.append(ref, kd, "k", table, lens, offs)
        R.append(ref, vd, "v", table, lens, offs)
        check_cache(cache, ref, table, lens, offs, lens)
        # read back whole, and the last rows alone
        whole = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
        for o in (whole, offs):
            gk, gv = cache.gather(tb, ln, dev(o), rows=int(o[-1]), dtype=DT[dtype])
            for got, which in ((gk, "k"), (gv, "v")):
                want = [R.tokens(ref, which, table[s], lens[s] - (o[s + 1] - o[s]), lens[s]) for s in range(len(lens))]
                want = np.concatenate(want)
                tol = np.abs(want) * 2.0 ** (-24 if dtype == "fp32" else -8)
                assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
    assert status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_token_by_token_append_grows_the_scale(fmt):
    """A page filled one token at a time, its magnitudes growing, shrinking, zero and not finite."""
    rng = np.random.default_rng(3)
    cache = KvCache(2, 2, 64, 32, fmt)
    ref = R.Paged(cache)
    table, offs = np.array([[1]], np.int32), np.array([0, 1], np.int32)
    widths = [0.0, 1e-3, 2e-3, 1.0, 0.5, 300.0, 1e-30, 0.0, 1e30, 2.0] + [1.0] * 22
    for t, w in enumerate(widths):
        x = rng.normal(size=(1, 2, 64)) * w
        if t in (4, 12):
            x[0, 0, 3], x[0, 1, 5], x[0, 1, 6] = np.inf, -np.inf, np.nan
        xt = torch.from_numpy(x.astype(np.float32))
        lens = np.array([t + 1], np.int32)
        cache.append(xt.to(DEV), (2 * xt).to(DEV), dev(table), dev(lens))
        R.append(ref, xt.double().numpy(), "k", table, lens, offs)
        R.append(ref, 2 * xt.double().numpy(), "v", table, lens, offs)
        check_cache(cache, ref, table, lens, offs, lens)
    assert status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantisation_error_is_half_a_step(fmt):
    rng = np.random.default_rng(9)
    cache = KvCache(4, 1, 128, 64, fmt)
    x, xd = draw(rng, (256, 1, 128), "fp32")
    table, lens = dev(np.array([[2, 0, 3, 1]], np.int32)), dev(np.array([256], np.int32))
    offs = dev(np.array([0, 256], np.int32))
    cache.append(x, x, table, lens, offs)
    k, v = cache.gather(table, lens, offs, rows=256, dtype=torch.float32)
    assert torch.equal(k, v)
    err = np.abs(k.double().cpu().numpy() - xd)
    s = np.repeat(cache.k_scales.cpu().double().numpy()[[2, 0, 3, 1], 0], 64)[:, None, None]
    # int8: half a step of the scale; e4m3: half a step of three mantissa bits, or of the least subnormal (2^-9 s)
    bound = s * 0.5 if fmt == "int8" else np.maximum(np.abs(xd) * 2.0 ** -4, s * 2.0 ** -10)
    assert np.all(err <= bound * (1 + 2.0 ** -20))


def test_ties_round_to_even():
    """amax 127 gives scale 1: halves are exact ties, which fp32 division keeps."""
    cache = KvCache(1, 1, 64, 16, "int8")
    x = torch.arange(64, dtype=torch.float32, device=DEV).sub_(31.5)
    x[0] = 127.0
    x = x.view(1, 1, 64)
    cache.append(x, x, dev(np.zeros((1, 1), np.int32)), dev(np.ones(1, np.int32)))
    want = torch.round(x.view(-1))
    assert torch.equal(cache.k_pages[0, 0, 0, 0, 0].float(), want)
    assert torch.equal(cache.v_pages[0, 0, 0, :, 0, :, 0].reshape(-1).float(), want)


def test_cache_errors_are_recorded_and_skipped():
    rng = np.random.default_rng(1)
    cache = KvCache(6, 2, 64, 16, "int8")
    R.random_codes(rng, cache)
    before = [t.clone() for t in (cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales)]
    x = torch.randn((4, 2, 64), device=DEV)

    def run(table, lens, offs):
        status()
        tb, ln, of = (dev(np.array(a, np.int32)) for a in (table, lens, offs))
        cache.append(x, x, tb, ln, of)
        st = device_status()
        k, v = cache.gather(tb, ln, of, rows=4, dtype=torch.float32,
                            k_out=torch.full((4, 2, 64), 7.0, device=DEV), v_out=torch.full((4, 2, 64), 7.0, device=DEV))
        assert device_status()[0] == st[0]
        q = torch.randn((4, 4, 64), device=DEV)
        o = cache.attention(q, tb, ln, of, out=torch.full((4, 4, 64), 7.0, device=DEV))
        assert device_status()[0] == st[0]
        return st, k, o

    # (status, sequence) and what comes back
    st, k, o = run([[0, 1], [2, 3]], [17, 40], [0, 2, 4])  # past max_pages
    assert st == (11, 1) and bool((k[2:] == 7).all()) and bool((o[2:] == 0).all()) and not bool((o[:2] == 0).all())
    st, k, o = run([[0, 1], [2, 3]], [1, 20], [0, 2, 4])  # more rows than tokens
    assert st == (8, 0) and bool((k[:2] == 7).all()) and bool((o[:2] == 0).all())
    st, k, o = run([[0, 1], [2, 3]], [20, 20], [0, 2, 5])  # offsets past the rows
    assert st == (8, 1) and bool((k[2:] == 7).all())
    st, k, o = run([[0, 1], [2, 3]], [20, -4], [0, 2, 4])  # negative length
    assert st == (11, 1) and bool((o[2:] == 0).all())
    for t, b in zip((cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales), before):
        assert torch.equal(t.view(torch.uint8)[4:], b.view(torch.uint8)[4:])
    st, k, o = run([[0, 6], [2, -1]], [20, 20], [0, 2, 4])  # table entries out of range: read as zeros
    assert st[0] == 11 and st[1] in (0, 1) and bool((k == 0).all()) and bool(torch.isfinite(o).all())


# ---------------------------------------------------------------- attention

def bounds(dtype, ref, lse, spread, score, n, vmax):
    rest = 2.0 ** -20 * (score + 16)
    if dtype == "bf16":
        tol = 2.0 ** -8 * np.abs(ref) + (spread * (2.0 ** -11 + rest) + n * 2.0 ** -25 * vmax)[..., None]
    else:
        tol = 2.0 ** -23 * np.abs(ref) + (spread * (2.0 ** -21 + rest) + n * 2.0 ** -36 * vmax)[..., None]
    return tol, rest


def check_attention(cache, rng, dtype, Hq, news, befores, table, lens, offs, causal=True, window=0, scale=None, q_width=1.0,
                    max_queries=None, ref=None, use_offsets=True, pad=16):
    ref = ref or R.Paged(cache)
    T, D = int(offs[-1]), cache.head_dim
    q, qd = draw(rng, (T, Hq, D), dtype, q_width, pad=pad)
    sm = D ** -0.5 if scale is None else scale
    out, lse = cache.attention(q, dev(table), dev(lens), dev(offs) if use_offsets else None, causal=causal, window=window,
                               scale=scale, return_lse=True, max_queries=max_queries or max(list(news) + [1]))
    want, wl, spread, score = R.attention(ref, qd, table, lens, offs, np.float32(sm).astype(np.float64), causal, window)
    assert status() == 0
    vmax = np.nanmax(np.abs(ref.v) * ref.vs[:, :, None, None]) if ref.v.size else 0.0
    tol, ltol = bounds(dtype, want, wl, spread, score, max(lens), vmax)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    err = np.abs(got - want)
    assert np.all(err <= tol), f"out: worst {np.nanmax(err / np.maximum(tol, 1e-300)):.3g} of its tolerance"
    np.testing.assert_array_equal(np.isneginf(gl), np.isneginf(wl))
    fin = np.isfinite(wl)
    assert np.all(np.abs(gl - wl)[fin] <= ltol[fin])
    return out, lse


def setup(seed, news, befores, page, fmt, H, D, **kw):
    rng = np.random.default_rng(seed)
    table, lens, offs, num = R.make_batch(rng, news, befores, page, **kw)
    cache = KvCache(num, H, D, page, fmt)
    R.random_codes(rng, cache)
    return rng, cache, table, lens, offs


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page,D,H,G", [(16, 128, 2, 8), (32, 64, 1, 1), (64, 128, 1, 5), (128, 64, 3, 4), (16, 64, 2, 16),
                                        (32, 128, 1, 12), (64, 64, 1, 17), (16, 128, 1, 64)])
def test_attention_decode(dtype, fmt, page, D, H, G):
    news, befores = [1] * 7, [0, 15, 16, 63, 130, 257, 700]
    rng, cache, table, lens, offs = setup(page + D + G, news, befores, page, fmt, H, D)
    check_attention(cache, rng, dtype, H * G, news, befores, table, lens, offs, use_offsets=False)
    check_attention(cache, rng, dtype, H * G, news, befores, table, lens, offs, q_width=4.0, window=50)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt,page,D,H,G,window,causal", [
    ("int8", 16, 128, 2, 8, 0, True), ("e4m3", 32, 64, 1, 4, 0, True), ("int8", 64, 128, 1, 3, 33, True),
    ("e4m3", 128, 128, 2, 1, 0, False), ("int8", 32, 64, 2, 5, 20, False), ("e4m3", 16, 64, 1, 32, 7, True),
])
def test_attention_several_queries(dtype, fmt, page, D, H, G, window, causal):
    for news, befores in (([4] * 3, [0, 61, 200]), ([2, 0, 7, 1], [5, 9, 0, 90]), ([37, 130], [0, 45]), ([1, 300], [600, 0])):
        rng, cache, table, lens, offs = setup(page + D + G + len(news), news, befores, page, fmt, H, D)
        check_attention(cache, rng, dtype, H * G, news, befores, table, lens, offs, causal, window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("news,befores,page,D,H,G,window,causal", [
    ([17], [0], 16, 128, 1, 1, 0, True), ([40, 3, 1], [5, 70, 300], 16, 128, 2, 4, 0, True),
    ([33], [130], 32, 64, 3, 5, 20, True), ([50, 20], [0, 11], 64, 128, 1, 8, 0, False), ([100], [400], 128, 64, 1, 4, 90, False),
])
def test_attention_several_queries_in_small_tables(fmt, news, befores, page, D, H, G, window, causal):
    """bf16, more than 16 query rows a sequence, tables with little room: several tiles of rows of the decode kernel."""
    rng, cache, table, lens, offs = setup(61 + D + G, news, befores, page, fmt, H, D, room=0)
    check_attention(cache, rng, "bf16", H * G, news, befores, table, lens, offs, causal=causal, window=window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_long_and_split(dtype, fmt):
    """One long sequence beside short ones: its keys are split over the machine and joined."""
    news, befores = [1, 1, 1], [20000, 3, 5000]
    rng, cache, table, lens, offs = setup(11, news, befores, 64, fmt, 2, 128)
    a = check_attention(cache, rng, dtype, 16, news, befores, table, lens, offs, q_width=2.0)
    b = check_attention(cache, np.random.default_rng(0), dtype, 16, news, befores, table, lens, offs, window=9000)
    assert a[0].shape == b[0].shape


def test_attention_is_deterministic():
    news, befores = [1] * 5 + [9], [7000, 20, 900, 0, 3000, 4000]
    rng, cache, table, lens, offs = setup(2, news, befores, 32, "int8", 4, 128)
    q = torch.randn((int(offs[-1]), 32, 128), device=DEV).bfloat16()
    args = (q, dev(table), dev(lens), dev(offs))
    a = cache.attention(*args, max_queries=9, return_lse=True)
    for _ in range(4):
        b = cache.attention(*args, max_queries=9, return_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n", [1, 40])
def test_attention_padding_rows(n):
    """Sequences of length 0 and rows without a key give 0 and -inf; rows outside every sequence stay as they are."""
    rng, cache, table, lens, offs = setup(4, [n, n, n], [100, 0, 31], 16, "int8", 1, 128)
    lens[1] = 0
    q, _ = draw(rng, (3 * n + 2, 8, 128), "bf16")
    out = torch.full_like(q, 7.0)
    lse = torch.full((3 * n + 2, 8), 7.0, device=DEV)
    cache.attention(q, dev(table), dev(lens), dev(offs), out=out, lse=lse, max_queries=n)
    assert status() == 0
    assert bool((out[n:2 * n] == 0).all()) and bool(torch.isneginf(lse[n:2 * n]).all())
    assert bool((out[3 * n:] == 7).all()) and bool((lse[3 * n:] == 7).all())
    assert bool(torch.isfinite(lse[:n]).all()) and bool(torch.isfinite(out).all())
    # a sequence with more rows than max_queries allows is skipped, and said
    if n > 1:
        cache.attention(q, dev(table), dev(lens), dev(offs), out=out, max_queries=n - 1)
        assert device_status()[0] == 8 and bool((out[:n] == 0).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype,news,befores", [("bf16", [1, 1], [37, 66]), ("bf16", [40, 70], [5, 33]), ("fp32", [3, 2], [37, 66])])
def test_attention_ignores_what_lies_past_the_end(fmt, dtype, news, befores):
    """Codes past a sequence's last token, NaN among them, and other sequences' pages do not reach the result."""
    rng, cache, table, lens, offs = setup(8, news, befores, 64, fmt, 2, 64)
    ref = R.Paged(cache)
    clean = check_attention(cache, np.random.default_rng(1), dtype, 8, news, befores, table, lens, offs, ref=ref)
    used = {}
    for s in range(2):
        for j in range(lens[s]):
            used.setdefault(int(table[s][j // 64]), set()).add(j % 64)
    bad = 0x7F if fmt == "e4m3" else 0x80
    kp, vp = cache.k_pages.view(torch.uint8).cpu(), cache.v_pages.view(torch.uint8).cpu()
    for page in range(cache.num_pages):
        for t in range(64):
            if t not in used.get(page, ()):
                kp[page, :, t // 16, :, t % 16] = bad
                vp[page, :, t // 16, :, t % 16 // 4, :, t % 4] = bad
    cache.k_pages.view(torch.uint8).copy_(kp)
    cache.v_pages.view(torch.uint8).copy_(vp)
    unused = [p for p in range(cache.num_pages) if p not in used]
    cache.k_scales[unused] = float("nan")
    cache.v_scales[unused] = float("inf")
    again = check_attention(cache, np.random.default_rng(1), dtype, 8, news, befores, table, lens, offs, ref=ref)
    assert torch.equal(clean[0], again[0]) and torch.equal(clean[1], again[1])


@pytest.mark.parametrize("n", [1, 48])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_scales_far_apart(dtype, n):
    """Pages of zeros (scale 0), and neighbouring pages whose scales differ by many orders."""
    rng, cache, table, lens, offs = setup(21, [n], [200], 16, "int8", 2, 128)
    pages = [int(p) for p in table[0] if p >= 0]
    for i, p in enumerate(pages):
        f = [1.0, 1e-4, 0.0, 30.0, 1e-8][i % 5]
        cache.v_scales[p] = f
        cache.k_scales[p] *= [1.0, 0.0, 1e-6, 1.0, 0.5][i % 5]
        if f == 0.0:
            cache.v_pages[p] = 0
        if i % 5 == 1:
            cache.k_pages[p] = 0
    check_attention(cache, rng, dtype, 8, [n], [200], table, lens, offs)
    # a sequence whose V is zero throughout: its softmax still sums to one
    cache.v_scales.zero_()
    out, lse = check_attention(cache, rng, dtype, 8, [n], [200], table, lens, offs)
    assert bool((out == 0).all())


@pytest.mark.parametrize("n", [1, 33])
@pytest.mark.parametrize("width,scale", [(1e-6, 0.08), (1e4, 1e-5), (60.0, 1.0), (1e30, 1e-31)])
def test_attention_query_ranges(n, width, scale):
    for dtype in ("bf16", "fp32"):
        rng, cache, table, lens, offs = setup(31, [n], [90], 32, "e4m3", 1, 64)
        check_attention(cache, rng, dtype, 4, [n], [90], table, lens, offs, q_width=width, scale=scale)


@pytest.mark.parametrize("window,room", [(0, 2048), (30, 2048), (30, 0)])
@pytest.mark.parametrize("dtype,n,before,D,page", [("bf16", 1, 100, 128, 16), ("bf16", 2, 100, 128, 16), ("bf16", 4, 5000, 64, 64),
                                                   ("fp32", 3, 100, 128, 32), ("bf16", 40, 100, 128, 16), ("bf16", 150, 100, 64, 128),
                                                   ("bf16", 70, 3000, 128, 64)])
def test_attention_nan_values_reach_the_rows_that_see_them(dtype, n, before, D, page, window, room):
    """NaN codes of V (e4m3): NaN in that dimension for the rows that see the token, and nothing else changes."""
    rng, cache, table, lens, offs = setup(51 + n, [n, 3], [before, 9], page, "e4m3", 2, D, room=room)
    L, G = before + n, 4
    bad = [(L - 1, 0, 3, 0x7F), (L - n // 2 - 1, 1, D - 1, 0xFF), (before - 20, 0, 33, 0x7F), (before - 29, 1, 0, 0xFF)]
    q, _ = draw(rng, (n + 3, 2 * G, D), dtype)

    def run(codes):
        vp = cache.v_pages.view(torch.uint8).cpu()
        for (t, h, d, _), c in zip(bad, codes):
            vp[int(table[0][t // page]), h, t % page // 16, d // 4, t % 16 // 4, d % 4, t % 4] = c
        cache.v_pages.view(torch.uint8).copy_(vp)
        return cache.attention(q, dev(table), dev(lens), dev(offs), window=window, return_lse=True, max_queries=max(n, 3))

    clean, clean_lse = run([0] * len(bad))
    out, lse = run([c for *_, c in bad])
    want = torch.zeros((n + 3, 2 * G, D), dtype=torch.bool)
    for i in range(n):
        for t, h, d, _ in bad:
            if t <= before + i and (window == 0 or t > before + i - window):
                want[i, h * G:(h + 1) * G, d] = True
    want = want.to(DEV)
    assert status() == 0 and bool(torch.isfinite(clean).all())
    assert torch.equal(torch.isnan(out), want)
    assert torch.equal(out[~want], clean[~want]) and torch.equal(lse, clean_lse)


def test_attention_nan_and_infinite_queries_stay_in_their_row():
    for n in (2, 40):
        rng, cache, table, lens, offs = setup(41, [n, n], [50, 60], 16, "int8", 1, 128)
        q, _ = draw(rng, (2 * n, 8, 128), "bf16")
        good = cache.attention(q, dev(table), dev(lens), dev(offs), max_queries=n)
        q[1, 3, 7] = float("nan")
        q[0, 5, 0] = float("inf")
        out = cache.attention(q, dev(table), dev(lens), dev(offs), max_queries=n)
        assert bool(torch.isnan(out[1, 3]).all()) and bool(torch.isnan(out[0, 5]).any())
        keep = torch.ones((2 * n, 8), dtype=torch.bool, device=DEV)
        keep[1, 3] = keep[0, 5] = False
        assert torch.equal(out[keep], good[keep])


def test_calls_on_another_stream_and_in_a_graph():
    rng, cache, table, lens, offs = setup(51, [1] * 4, [100, 40, 16, 300], 16, "e4m3", 2, 128)
    tb, ln = dev(table), dev(lens)
    k, _ = draw(rng, (4, 2, 128), "bf16")
    q, _ = draw(rng, (4, 16, 128), "bf16")
    cos, sin = rope_tables(512, 128, device=DEV)
    pos = ln - 1

    def step(stream=None):
        qr, kr = rope(q, k, cos, sin, pos, stream=stream)
        cache.append(kr, k, tb, ln, stream=stream)
        return cache.attention(qr, tb, ln, stream=stream)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    captured.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, want)
    assert status() == 0


def test_offsets_past_32_bits():
    """Pages past 4 GiB of codes."""
    H, D, page = 8, 128, 128
    num = (1 << 32) // (H * D * page) + 40  # K codes alone pass 4 GiB
    cache = KvCache(num, H, D, page, "int8")
    rng = np.random.default_rng(6)
    ids = np.array([[num - 1, 3, num - 2], [num - 30, num - 31, 0]], np.int32)
    lens, offs = np.array([300, 129], np.int32), np.array([0, 300, 429], np.int32)
    k, kd = draw(rng, (429, H, D), "bf16")
    v, vd = draw(rng, (429, H, D), "bf16")
    cache.append(k, v, dev(ids), dev(lens), dev(offs))
    gk, gv = cache.gather(dev(ids), dev(lens), dev(offs), rows=429, dtype=torch.float32)
    step = 4.0 * np.abs(kd).max() / 127
    assert np.all(np.abs(gk.double().cpu().numpy() - kd) <= step) and np.all(np.abs(gv.double().cpu().numpy() - vd) <= step)
    small = KvCache(6, H, D, page, "int8")
    order = ids.reshape(-1)
    for a, b in ((small.k_pages, cache.k_pages), (small.v_pages, cache.v_pages), (small.k_scales, cache.k_scales),
                 (small.v_scales, cache.v_scales)):
        a.copy_(b[torch.from_numpy(order.astype(np.int64)).to(DEV)])
    tb = dev(np.arange(6, dtype=np.int32).reshape(2, 3))
    q = torch.randn((429, 16, D), device=DEV).bfloat16()
    for rows, o in ((429, offs), (2, None)):
        a = cache.attention(q[:rows], dev(ids), dev(lens), None if o is None else dev(o), max_queries=300 if o is not None else 1)
        b = small.attention(q[:rows], tb, dev(lens), None if o is None else dev(o), max_queries=300 if o is not None else 1)
        assert torch.equal(a, b)
    assert status() == 0


def test_binding_refusals():
    cache = KvCache(4, 2, 128, 16, "int8")
    tb, ln = torch.zeros((2, 2), dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    x = torch.zeros((2, 2, 128), device=DEV)
    with pytest.raises(ValueError):
        cache.append(x[..., :64], x, tb, ln)
    with pytest.raises(ValueError):
        cache.append(x, x, tb.long(), ln)
    with pytest.raises(ValueError):
        cache.append(x, x, tb, ln, offsets=ln)
    with pytest.raises(TypeError):
        cache.append(x.half(), x.half(), tb, ln)
    with pytest.raises(ValueError):
        cache.gather(tb, ln, offsets=torch.zeros(3, dtype=torch.int32, device=DEV))
    with pytest.raises(LoraError):
        cache.attention(torch.zeros((2, 3, 128), device=DEV), tb, ln)
    with pytest.raises(LoraError):
        cache.attention(x, tb, ln, workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        KvCache(4, 2, 128, 16, "int4")
    with pytest.raises(LoraError):
        KvCache(4, 2, 128, 8, "int8").append(x, x, tb, ln)
    with pytest.raises(ValueError):
        rope(x, None, torch.zeros((4, 64), device=DEV), torch.zeros((4, 32), device=DEV), ln)
