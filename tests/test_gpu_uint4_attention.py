"""GPU parity of attention over the 4-bit cache with a plain float64 restatement.

Tolerances as derived at the head of test_gpu_attention.py, with |v| = |scale code| + |least| (the parts enter the
products apart), per row:
    bf16: 2^-8 |o| + A (2^-11 + 2^-20 (S + 16)) + n 2^-25 V;  fp32: 2^-23 |o| + A (2^-21 + 2^-20 (S + 16)) + n 2^-36 V;
    lse: 2^-20 (S + 16).
(p' = p scale has 11 or 22 bits; the least values' sums are fp32.)  Where a call takes the kernel for many queries, V
enters rounded to f16, and without lse K too: the restatement rounds them so too, and |v| is that value's."""

import numpy as np
import pytest
import torch

import attention_reference as R
import uint4_reference as U
from adapter_gemm_linear_gb300 import KvCache, arm_test_wait_timeout, device_status, rope_tables
from test_gpu_attention import bounds, dev, draw, status
from test_gpu_attention_layouts import CALLS, LAYOUTS, laid_out

pytestmark = pytest.mark.gpu

DEV = "cuda"


def setup(seed, news, befores, page, H, D, **kw):
    rng = np.random.default_rng(seed)
    table, lens, offs, num = R.make_batch(rng, news, befores, page, **kw)
    cache = KvCache(num, H, D, page, "uint4", device=DEV)
    U.random_cache(rng, cache)
    return rng, cache, table, lens, offs


def many_queries(dtype, T, cache, G, table, max_queries):
    """Which kernel: the rule of the library's host side."""
    n = max_queries * G
    if dtype != "bf16" or n <= (32 if cache.head_dim == 64 else 16):
        return False
    S, sms = table.shape[0], torch.cuda.get_device_properties(0).multi_processor_count
    row_tiles = min(S * ((n + 15) // 16), T * G / 16 + S)
    return row_tiles * cache.num_heads * ((table.shape[1] * cache.page_tokens + 127) / 128) > 8 * sms


def check(cache, rng, dtype, Hq, news, table, lens, offs, causal=True, window=0, scale=None, q_width=1.0, ref=None, use_offsets=True,
          q=None):
    ref = ref or U.Paged4(cache)
    T, D = int(offs[-1]), cache.head_dim
    q, qd = draw(rng, (T, Hq, D), dtype, q_width, pad=16) if q is None else q
    sm = D ** -0.5 if scale is None else scale
    most = max(list(news) + [1])
    out, lse = cache.attention(q, dev(table), dev(lens), dev(offs) if use_offsets else None, causal=causal, window=window,
                               scale=scale, return_lse=True, max_queries=most)
    assert status() == 0
    many = many_queries(dtype, T, cache, Hq // cache.num_heads, table, most)
    rounded = "v" if many else ""
    want, wl, spread, score, vmax = U.attention(ref, qd, table, lens, offs, np.float32(sm).astype(np.float64), causal, window, rounded)
    tol, ltol = bounds(dtype, want, wl, spread, score, max(lens), vmax)
    if many:  # and without lse
        alone = cache.attention(q, dev(table), dev(lens), dev(offs) if use_offsets else None, causal=causal, window=window,
                                scale=scale, max_queries=most)
        want2, wl2, spread2, score2, vmax2 = U.attention(ref, qd, table, lens, offs, np.float32(sm).astype(np.float64), causal, window, "kv")
        err = np.abs(alone.double().cpu().numpy() - want2)
        tol2 = bounds(dtype, want2, wl2, spread2, score2, max(lens), vmax2)[0]
        assert np.all(err <= tol2), f"out without lse: worst {np.nanmax(err / np.maximum(tol2, 1e-300)):.3g} of its tolerance"
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    err = np.abs(got - want)
    assert np.all(err <= tol), f"out: worst {np.nanmax(err / np.maximum(tol, 1e-300)):.3g} of its tolerance"
    np.testing.assert_array_equal(np.isneginf(gl), np.isneginf(wl))
    fin = np.isfinite(wl)
    assert np.all(np.abs(gl - wl)[fin] <= ltol[fin]), f"lse: worst {np.max(np.abs(gl - wl)[fin] / ltol[fin]):.3g}"
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("page,D,H,G", [(16, 128, 2, 8), (32, 64, 1, 1), (64, 128, 1, 5), (128, 64, 3, 4), (16, 64, 2, 16),
                                        (32, 128, 1, 12), (64, 64, 1, 17), (16, 128, 1, 64)])
def test_decode(dtype, page, D, H, G):
    news, befores = [1] * 7, [0, 15, 16, 63, 130, 257, 700]
    rng, cache, table, lens, offs = setup(page + D + G, news, befores, page, H, D)
    check(cache, rng, dtype, H * G, news, table, lens, offs, use_offsets=False)
    check(cache, rng, dtype, H * G, news, table, lens, offs, q_width=4.0, window=50)


@pytest.mark.parametrize("room", [0, 2048])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("page,D,H,G,window,causal", [
    (16, 128, 2, 8, 0, True), (32, 64, 1, 4, 0, True), (64, 128, 1, 3, 33, True), (128, 128, 2, 1, 0, False),
    (32, 64, 2, 5, 20, False), (16, 64, 1, 32, 7, True),
])
def test_several_queries(dtype, page, D, H, G, window, causal, room):
    for news, befores in (([4] * 3, [0, 61, 200]), ([2, 0, 7, 1], [5, 9, 0, 90]), ([37, 130], [0, 45]), ([1, 300], [600, 0])):
        rng, cache, table, lens, offs = setup(page + D + G + len(news), news, befores, page, H, D, room=room)
        check(cache, rng, dtype, H * G, news, table, lens, offs, causal, window)


@pytest.mark.parametrize("n,G", [(17, 1), (33, 1), (9, 5), (127, 1), (43, 3), (130, 1), (37, 7), (255, 1), (259, 1), (20, 13)])
@pytest.mark.parametrize("D", [64, 128])
def test_row_tiles_that_end_inside_a_warp(n, G, D):
    news, befores = [n, n, 1], [0, 2000, 300]
    rng, cache, table, lens, offs = setup(n * G, news, befores, 16, 1, D)
    check(cache, rng, "bf16", G, news, table, lens, offs)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_long_and_split(dtype):
    """One long sequence beside short ones: its keys are split over the machine and joined."""
    news, befores = [1, 1, 1], [20000, 3, 5000]
    rng, cache, table, lens, offs = setup(11, news, befores, 64, 2, 128)
    check(cache, rng, dtype, 16, news, table, lens, offs, q_width=2.0)
    check(cache, np.random.default_rng(0), dtype, 16, news, table, lens, offs, window=9000)


def test_many_sequences():
    """More items than CTAs, lengths of one token up, an odd number of tiles, every order of lengths."""
    rng = np.random.default_rng(9)
    befores = [int(x) for x in np.exp(rng.uniform(0, 7, 200))]
    for D, G in ((128, 8), (64, 4)):
        rng, cache, table, lens, offs = setup(D, [1] * 200, befores, 16, 2, D)
        check(cache, rng, "bf16", 2 * G, [1] * 200, table, lens, offs, use_offsets=False)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("fp32", 64)])
def test_more_items_than_are_described_at_once(dtype, D):
    """Some hundred items a CTA, of one tile to three, and one of many among them."""
    rng = np.random.default_rng(D)
    befores = [int(x) for x in rng.integers(0, 40, 6000)]
    befores[1234] = 3000
    rng, cache, table, lens, offs = setup(D + 1, [1] * 6000, befores, 16, 8, D)
    check(cache, rng, dtype, 8, [1] * 6000, table, lens, offs, use_offsets=False)


@pytest.mark.parametrize("n", [1, 40])
def test_padding_rows(n):
    """Sequences of length 0 give 0 and -inf; rows outside every sequence stay as they are."""
    rng, cache, table, lens, offs = setup(4, [n, n, n], [100, 0, 31], 16, 1, 128)
    lens[1] = 0
    q, _ = draw(rng, (3 * n + 2, 8, 128), "bf16")
    out = torch.full_like(q, 7.0)
    lse = torch.full((3 * n + 2, 8), 7.0, device=DEV)
    cache.attention(q, dev(table), dev(lens), dev(offs), out=out, lse=lse, max_queries=n)
    assert status() == 0
    assert bool((out[n:2 * n] == 0).all()) and bool(torch.isneginf(lse[n:2 * n]).all())
    assert bool((out[3 * n:] == 7).all()) and bool((lse[3 * n:] == 7).all())
    assert bool(torch.isfinite(lse[:n]).all()) and bool(torch.isfinite(out).all())
    if n > 1:
        cache.attention(q, dev(table), dev(lens), dev(offs), out=out, max_queries=n - 1)
        assert device_status()[0] == 8 and bool((out[:n] == 0).all())


def test_bad_tables_read_as_zeros():
    for n in (1, 60):
        rng, cache, table, lens, offs = setup(14, [n, n], [100, 90], 16, 2, 64)
        table[0, 2], table[1, 1] = -1, cache.num_pages
        q, qd = draw(rng, (2 * n, 8, 64), "bf16")
        status()
        out, lse = cache.attention(q, dev(table), dev(lens), dev(offs), max_queries=n, return_lse=True)
        st, s = device_status()
        assert st == 11 and s in (0, 1)
        rounded = "v" if many_queries("bf16", 2 * n, cache, 4, table, n) else ""
        want, wl, spread, score, vmax = U.attention(U.Paged4(cache), qd, table, lens, offs, 0.125, True, 0, rounded)
        tol, ltol = bounds("bf16", want, wl, spread, score, max(lens), vmax)
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)
        assert np.all(np.abs(lse.double().cpu().numpy() - wl) <= ltol)


@pytest.mark.parametrize("dtype,news,befores", [("bf16", [1, 1], [37, 66]), ("bf16", [40, 70], [5, 33]), ("fp32", [3, 2], [37, 66])])
@pytest.mark.parametrize("room", [0, 2048])
def test_what_lies_past_the_end_is_ignored(dtype, news, befores, room):
    """Scales that are NaN and codes past a sequence's last token, and other sequences' pages, do not reach the result."""
    rng, cache, table, lens, offs = setup(8, news, befores, 64, 2, 64, room=room)
    ref = U.Paged4(cache)
    clean = check(cache, np.random.default_rng(1), dtype, 8, news, table, lens, offs, ref=ref)
    used = {}
    for s in range(2):
        for j in range(lens[s]):
            used.setdefault(int(table[s][j // 64]), set()).add(j % 64)
    for name in ("k", "v"):
        x = getattr(cache, name + "_pages").cpu().numpy().reshape(cache.num_pages, 2, 4, -1)
        sc = getattr(cache, name + "_scales").cpu().numpy()
        byte, high = ref.where[name]
        for page in range(cache.num_pages):
            for t in range(64):
                if t not in used.get(page, ()):
                    x[page, :, t // 16][:, byte[t % 16]] = 0xFF
                    sc[page, :, t // 16, :, t % 16] = [np.nan, np.inf] if t % 2 else [np.inf, np.nan]
        getattr(cache, name + "_pages").view(-1).copy_(torch.from_numpy(x.reshape(-1)))
        getattr(cache, name + "_scales").copy_(torch.from_numpy(sc))
    again = check(cache, np.random.default_rng(1), dtype, 8, news, table, lens, offs, ref=ref)
    assert torch.equal(clean[0], again[0]) and torch.equal(clean[1], again[1])


KINDS = ["zeros", "zero first", "least", "largest", "rising", "falling", "any", "huge at the end", "least values alone"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,n,before,page,D", [("bf16", 1, 900, 16, 128), ("bf16", 2, 900, 32, 64), ("fp32", 2, 600, 16, 64),
                                                  ("fp32", 1, 6000, 64, 128), ("bf16", 48, 700, 16, 128), ("bf16", 200, 4000, 64, 64)])
def test_scales_of_v_anywhere(kind, dtype, n, before, page, D):
    """V's scales from 2^-24 to 2^12, in any order, and none (values within f16's range, as the format has them); each row's
    tolerance by the V that it sees."""
    rng, cache, table, lens, offs = setup(before + n, [n, 3], [before, 40], page, 2, D)
    sc = np.zeros(tuple(cache.v_scales.shape), np.float64)
    for s in range(2):
        L = int(lens[s])
        for j in range(L):
            e = {"zeros": -np.inf, "zero first": -np.inf if j < L // 2 else -3, "least": -24, "largest": 12,
                 "rising": -24 + 36 * j / L, "falling": 12 - 36 * j / L, "any": rng.choice([-24, -np.inf, -12, -2, 5, 12]),
                 "huge at the end": 12 if j >= L - n else -20, "least values alone": -np.inf}[kind]
            least = -(7.5 + 1.5 * np.clip(rng.normal(), -2, 2)) * 2.0 ** e if np.isfinite(e) else 0.0
            if kind == "least values alone":
                least = rng.normal() * 100
            at = sc[int(table[s][j // page]), :, j % page // 16, :, j % 16]
            at[..., 0], at[..., 1] = 2.0 ** e, least
    cache.v_scales.copy_(torch.from_numpy(sc.astype(np.float16)))
    out, _ = check(cache, rng, dtype, 8, [n, 3], table, lens, offs, q_width=2.0)
    assert kind != "zeros" or bool((out == 0).all())


@pytest.mark.parametrize("n", [1, 33])
@pytest.mark.parametrize("width,scale", [(1e-6, 0.08), (1e4, 1e-5), (60.0, 1.0), (1e30, 1e-31)])
def test_query_ranges(n, width, scale):
    for dtype in ("bf16", "fp32"):
        rng, cache, table, lens, offs = setup(31, [n], [90], 32, 1, 64)
        check(cache, rng, dtype, 4, [n], table, lens, offs, q_width=width, scale=scale)


@pytest.mark.parametrize("k_size,spread", [(30.0, 0.3), (1e-4, 2.0), (3000.0, 1.0)])
@pytest.mark.parametrize("dtype,n", [("bf16", 1), ("fp32", 3), ("bf16", 70)])
def test_keys_of_any_size(dtype, n, k_size, spread):
    """Scores far apart (one key takes all) and nearly equal; growing along the sequence and shrinking."""
    for order in (1, -1):
        rng, cache, table, lens, offs = setup(77, [n, 2], [500, 333], 16, 2, 128)
        sc = cache.k_scales.cpu().numpy().astype(np.float64)
        for s in range(2):
            for j in range(int(lens[s])):
                sc[int(table[s][j // 16]), :, 0, :, j % 16] *= k_size * np.exp(spread * order * (j / lens[s] - 0.5)) / 8
        cache.k_scales.copy_(torch.from_numpy(sc.astype(np.float16)))
        check(cache, rng, dtype, 8, [n, 2], table, lens, offs, q_width=1.0)


def test_nan_and_infinite_queries_stay_in_their_row():
    for n in (2, 40):
        rng, cache, table, lens, offs = setup(41, [n, n], [50, 60], 16, 1, 128)
        q, _ = draw(rng, (2 * n, 8, 128), "bf16")
        good = cache.attention(q, dev(table), dev(lens), dev(offs), max_queries=n)
        q[1, 3, 7] = float("nan")
        q[0, 5, 0] = float("inf")
        out = cache.attention(q, dev(table), dev(lens), dev(offs), max_queries=n)
        assert bool(torch.isnan(out[1, 3]).all()) and bool(torch.isnan(out[0, 5]).any())
        keep = torch.ones((2 * n, 8), dtype=torch.bool, device=DEV)
        keep[1, 3] = keep[0, 5] = False
        assert torch.equal(out[keep], good[keep])


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype,news,befores,D,page", CALLS)
def test_layouts(layout, dtype, news, befores, D, page):
    rng, cache, table, lens, offs = setup(len(news) + D, news, befores, page, 2, D)
    q = draw(rng, (int(offs[-1]), 10, D), dtype)[0].contiguous()
    args = dev(table), dev(lens), dev(offs)
    want, lse = cache.attention(q, *args, max_queries=max(news), return_lse=True)
    view, whole, outside = laid_out(torch.zeros_like(q), LAYOUTS[(LAYOUTS.index(layout) + 1) % len(LAYOUTS)])
    got, lse2 = cache.attention(laid_out(q, layout)[0], *args, max_queries=max(news), out=view, return_lse=True)
    assert torch.equal(got, want) and torch.equal(lse2, lse) and bool((whole[outside] == 7).all())
    assert status() == 0


@pytest.mark.parametrize("dtype,news,befores,D,page", CALLS)
def test_repeats_itself_and_runs_in_a_graph(dtype, news, befores, D, page):
    """The same bits every time, from two graphs over one workspace too, with the lengths that are there when they are replayed."""
    rng, cache, table, lens, offs = setup(3 * len(news) + D, news, befores, page, 2, D)
    q = draw(rng, (int(offs[-1]), 10, D), dtype)[0].contiguous()
    tb, ln, of = dev(table), dev(lens), dev(offs)
    space = torch.full((1 << 27,), 0x7F, dtype=torch.uint8, device=DEV)

    def call():
        return cache.attention(q, tb, ln, of, max_queries=max(news), return_lse=True, workspace=space)

    want = call()
    for _ in range(5):
        again = call()
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    shorter = dev(np.maximum(lens - 3, np.diff(offs)).astype(np.int32))
    want_shorter = cache.attention(q, tb, shorter, of, max_queries=max(news), return_lse=True)
    graphs, captured = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            captured.append(call())
    for lengths, w in ((ln.clone(), want), (shorter, want_shorter), (ln.clone(), want)):
        ln.copy_(lengths)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c in captured:
            assert torch.equal(c[0], w[0]) and torch.equal(c[1], w[1])
            c[0].fill_(7)
    assert status() == 0


@pytest.mark.parametrize("dtype,n,before,D", [("bf16", 1, 900, 128), ("fp32", 3, 3000, 64), ("bf16", 60, 100, 128), ("bf16", 300, 5000, 64),
                                             ("bf16", 17, 40000, 128)])
def test_waits_that_run_out_are_reported_and_the_next_call_is_right(dtype, n, before, D):
    rng, cache, table, lens, offs = setup(n + D, [n, 2], [before, 70], 32, 2, D)
    T = int(offs[-1])
    q, _ = draw(rng, (T, 8, D), dtype)
    args = dev(table), dev(lens), dev(offs)
    want = cache.attention(q, *args, max_queries=n + 1, return_lse=True)
    out = torch.full((T + 8, 8, D), 7.0, dtype=q.dtype, device=DEV)
    status()
    for limit in (5_000_000, 20_000_000):
        arm_test_wait_timeout(limit)
        cache.attention(q, *args, max_queries=n + 1, out=out[4:T + 4])
        st, site = device_status()
        assert st == 10 and 40 <= site <= 91, (st, site)
        assert bool((out[:4] == 7).all()) and bool((out[T + 4:] == 7).all())
        again = cache.attention(q, *args, max_queries=n + 1, return_lse=True)
        assert status() == 0
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_offsets_past_32_bits():
    """Pages past 4 GiB of codes."""
    H, D, page = 8, 128, 128
    num = (1 << 33) // (H * D * page) + 40  # K codes alone pass 4 GiB
    cache = KvCache(num, H, D, page, "uint4", device=DEV)
    rng = np.random.default_rng(6)
    ids = np.array([[num - 1, 3, num - 2], [num - 30, num - 31, 0]], np.int32)
    lens, offs = np.array([300, 129], np.int32), np.array([0, 300, 429], np.int32)
    k, kd = draw(rng, (429, H, D), "bf16")
    v, vd = draw(rng, (429, H, D), "bf16")
    cache.append(k, v, dev(ids), dev(lens), dev(offs))
    gk, gv = cache.gather(dev(ids), dev(lens), dev(offs), rows=429, dtype=torch.float32)
    small = KvCache(6, H, D, page, "uint4", device=DEV)
    tb = dev(np.arange(6, dtype=np.int32).reshape(2, 3))
    small.append(k, v, tb, dev(lens), dev(offs))
    sk, sv = small.gather(tb, dev(lens), dev(offs), rows=429, dtype=torch.float32)
    assert torch.equal(gk, sk) and torch.equal(gv, sv)
    q = torch.randn((429, 16, D), device=DEV).bfloat16()
    for rows, o in ((429, offs), (2, None)):
        a = cache.attention(q[:rows], dev(ids), dev(lens), None if o is None else dev(o), max_queries=300 if o is not None else 1)
        b = small.attention(q[:rows], tb, dev(lens), None if o is None else dev(o), max_queries=300 if o is not None else 1)
        assert torch.equal(a, b)
    assert status() == 0


def test_a_decoded_sequence_on_another_stream_and_in_a_graph():
    """Norms and positions, a token appended, attention: in turn, as a decode step runs them."""
    from adapter_gemm_linear_gb300 import norm_rope
    rng, cache, table, lens, offs = setup(51, [1] * 4, [100, 40, 16, 300], 16, 2, 128)
    tb, ln = dev(table), dev(lens)
    k, q = draw(rng, (4, 2, 128), "bf16")[0], draw(rng, (4, 16, 128), "bf16")[0]
    w = torch.rand((2, 128), device=DEV).bfloat16() + 0.5
    cos, sin = rope_tables(512, 128, device=DEV)
    pos = ln - 1

    def step(stream=None):
        qr, kr = norm_rope(q, k, w[0], w[1], cos, sin, pos, stream=stream)
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
    # and against the pieces: the cache's tokens are the turned keys, quantised
    ref = U.Paged4(cache)
    qr, kr = norm_rope(q, k, w[0], w[1], cos, sin, pos)
    check(cache, rng, "bf16", 16, [1] * 4, table, lens, offs, use_offsets=False, q=(qr, qr.double().cpu().numpy()))
    for s in range(4):
        page, t = int(table[s][(lens[s] - 1) // 16]), (lens[s] - 1) % 16
        codes, sc = U.quantise(kr[s].float().cpu().numpy().reshape(2, 2, 64))
        np.testing.assert_array_equal(ref.k[page, :, t], codes.reshape(2, 128))
    assert status() == 0
