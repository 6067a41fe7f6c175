"""Inputs at the edge of the cache's and attention's definitions
(include/lora_attention.h): values that are not finite, scales at both ends of
their range, probabilities far below the largest, and calls that overlap.

Reference: tests/attention_reference.py in float64, with its tolerances as
derived at the head of test_gpu_attention.py; where that reference does not
follow the header, the header's words are restated here."""

import numpy as np
import pytest
import torch

import attention_reference as R
from adapter_gemm_linear_gb300 import KvCache
from test_gpu_attention import DT, FORMATS, bounds, check_attention, dev, draw, setup, status

pytestmark = pytest.mark.gpu

DEV = "cuda"


# ---------------------------------------------------------------- rows that are not finite, first in their page

NAN, INF = float("nan"), float("inf")
LEAST = 2.0 ** -120


def first_row(kind, rng, D):
    x = np.zeros(D)
    if kind == "all nan":
        x[:] = NAN
    elif kind == "all inf":
        x[:] = np.where(rng.random(D) < 0.5, -INF, INF)
    elif kind == "one nan":
        x[D - 3] = NAN
    elif kind == "one inf":
        x[5] = -INF
    elif kind == "both":
        x[1], x[D // 2], x[D - 1] = NAN, INF, -INF
    return x


@pytest.mark.parametrize("kind", ["all nan", "all inf", "one nan", "one inf", "both", "zeros"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype,D,page", [("bf16", 128, 16), ("fp32", 64, 32), ("fp32", 128, 128), ("bf16", 64, 64)])
def test_rows_that_are_not_finite_first_in_their_page(kind, fmt, dtype, D, page):
    """NaN reads back as NaN (e4m3) or 0 (int8), an infinity as the largest code; and so, whole, with the page's other heads untouched."""
    rng = np.random.default_rng(D + page)
    for rows in (1, 3):  # alone, and with two rows of zeros after it
        cache = KvCache(3, 2, D, page, fmt)
        R.random_codes(rng, cache)
        x = np.zeros((rows, 2, D))
        x[0, 0] = first_row(kind, rng, D)
        x[:, 1] = 1.0
        t = torch.from_numpy(x).to(DT[dtype]).to(DEV)
        table, lens, offs = dev(np.array([[2]], np.int32)), dev(np.array([rows], np.int32)), dev(np.array([0, rows], np.int32))
        cache.append(t, t, table, lens, offs)
        got = cache.gather(table, lens, offs, rows=rows, dtype=torch.float32)
        top = 127.0 if fmt == "int8" else 448.0
        want = np.where(np.isnan(x), NAN if fmt == "e4m3" else 0.0, np.clip(x, -top * LEAST, top * LEAST))
        for y, scales in zip(got, (cache.k_scales, cache.v_scales)):
            np.testing.assert_array_equal(y.cpu().double().numpy()[:, 0], want[:, 0])
            assert float(scales[2, 0]) == (0.0 if kind == "zeros" else LEAST)
            assert bool((y[:, 1] == (1.0 if fmt == "e4m3" else y[0, 1, 0])).all()) and abs(float(y[0, 1, 0]) - 1.0) < 2.0 ** -22
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 40])
def test_a_nan_row_first_in_its_page_reaches_attention(dtype, n):
    """A K or V row that is NaN throughout, the first token of an e4m3 page: its key/value head's queries are NaN, the other's are not."""
    for which in "kv":
        rng = np.random.default_rng(n)
        table, lens, offs, num = R.make_batch(rng, [n], [16], 16)
        cache = KvCache(num, 2, 128, 16, "e4m3")
        x = rng.normal(size=(16 + n, 2, 128))
        bad = x.copy()
        bad[16, 0] = NAN
        k, v = (torch.from_numpy(y).to(DT[dtype]).to(DEV) for y in ((bad, x) if which == "k" else (x, bad)))
        tb, of = dev(table), dev(offs)
        # the page before, then the rows one by one: the bad one alone is the first of its page
        cache.append(k[:16], v[:16], tb, dev(lens - n), dev(np.array([0, 16], np.int32)))
        for i in range(n):
            cache.append(k[16 + i:17 + i], v[16 + i:17 + i], tb, dev(lens - n + i + 1))
        q = torch.randn((n, 8, 128), device=DEV).to(DT[dtype])
        out = cache.attention(q, tb, dev(lens), of, max_queries=n)
        assert bool(torch.isnan(out[:, :4]).all()) and bool(torch.isfinite(out[:, 4:]).all())
    assert status() == 0


# ---------------------------------------------------------------- scales of V at both ends of their range

def v_scales(kind, i, count, rng):
    """Of page i of `count` of a sequence, in log2."""
    if kind == "least":
        return -120.0
    if kind == "largest":
        return 108.0
    if kind == "least, then ordinary":
        return -120.0 if i < count // 2 else -6.0
    if kind == "ordinary, then least":
        return -6.0 if i < count // 2 else -120.0
    if kind == "rising":
        return -120.0 + 200.0 * i / count
    if kind == "falling":
        return 80.0 - 200.0 * i / count
    if kind == "zeros, then least":
        return -np.inf if i < count // 3 else -120.0
    return rng.choice([-120.0, -np.inf, -60.0, -20.0, 0.0, 30.0, 75.0])  # "any"


KINDS = ["least", "largest", "least, then ordinary", "ordinary, then least", "rising", "falling", "zeros, then least", "any"]


@pytest.mark.parametrize("k_growth", [1.0, 40.0, 0.02])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,fmt,n,before,page,D", [
    ("bf16", "int8", 1, 900, 16, 128), ("bf16", "e4m3", 2, 900, 32, 64), ("fp32", "int8", 2, 600, 16, 64),
    ("fp32", "e4m3", 1, 6000, 64, 128), ("bf16", "int8", 48, 700, 16, 128), ("bf16", "e4m3", 200, 4000, 64, 64),
])
def test_attention_with_v_scales_anywhere(kind, k_growth, dtype, fmt, n, before, page, D):
    """Scales from 2^-120 up, scores that grow or shrink along the sequence: the softmax's sum stays itself (lse), and so does the result."""
    rng, cache, table, lens, offs = setup(before + n, [n, 3], [before, 40], page, fmt, 2, D)
    for s in range(2):
        pages = [int(p) for p in table[s] if p >= 0]
        for i, p in enumerate(pages):
            scale = float(np.exp2(np.float32(v_scales(kind, i, len(pages), rng))))
            cache.v_scales[p] = scale
            if scale == 0.0:
                cache.v_pages[p] = 0
            cache.k_scales[p] *= k_growth ** (i / len(pages))
    check_attention(cache, rng, dtype, 8, [n, 3], [before, 40], table, lens, offs, q_width=1.0 if k_growth > 1 else 3.0)


# ---------------------------------------------------------------- probabilities far below the largest

def sink_and_tail(fmt, n, before, page, D, below, H=1):
    """A first key whose score is `below` (log2) above all others', which are equal; V of the first is zero but in dimension 0."""
    rng, cache, table, lens, offs = setup(int(before + below), [n], [before], page, fmt, H, D)
    kp = torch.zeros((cache.num_pages, H, page, D), dtype=torch.float32)
    first = int(table[0][0])
    kp[first, :, 0, 0] = 96.0
    vp = torch.from_numpy(rng.integers(4, 8, (cache.num_pages, H, page, D)).astype(np.float32) * 16)  # codes of both formats
    vp[first, :, 0] = 0.0
    vp[first, :, 0, 0] = 96.0
    tiles = page // 16
    cache.k_pages.copy_(kp.view(-1, H, tiles, 16, D // 64, 64).transpose(3, 4).to(cache.k_pages.dtype))
    cache.v_pages.copy_(vp.view(-1, H, tiles, 4, 4, D // 4, 4).permute(0, 1, 2, 5, 3, 6, 4).to(cache.v_pages.dtype))
    cache.k_scales.fill_(0.25)
    cache.v_scales.fill_(0.125)
    return cache, table, lens, offs


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("below", [20.4, 23.4, 26.4])
@pytest.mark.parametrize("dtype,n,before,page,D,start,seqs", [
    ("bf16", 1, 4000, 16, 128, 33, 1), ("bf16", 3, 30000, 64, 64, 33, 1), ("bf16", 20, 131072, 128, 64, 29, 1),
    ("bf16", 1, 4000, 16, 128, 33, 64), ("fp32", 2, 2000, 32, 64, 44, 64), ("bf16", 40, 4000, 16, 128, 29, 20),
    ("bf16", 20, 32768, 128, 64, 29, 20),
])
def test_a_long_tail_behind_a_dominant_key(fmt, below, dtype, n, before, page, D, start, seqs):
    """What many small probabilities add up to: off by their 11 (22) bits and by 2^-start of the largest each, no more.
    `seqs` sequences of the same pages (few CTAs an item: the tail is summed where the dominant key is)."""
    H = 1 if seqs == 1 else 8
    cache, table, lens, offs = sink_and_tail(fmt, n, before, page, D, below, H)
    q = torch.zeros((seqs * n, 4 * H, D), dtype=DT[dtype], device=DEV)
    q[..., 0] = 1.0
    scale = float(np.float32(below * np.log(2.0) / 24.0))
    out, lse = cache.attention(q, dev(np.repeat(table, seqs, 0)), dev(np.repeat(lens, seqs)),
                               dev(np.arange(seqs + 1, dtype=np.int32) * n), scale=scale, max_queries=n, return_lse=True)
    want, wl, _, score = R.attention(R.Paged(cache), q[:n].double().cpu().numpy(), table, lens, offs, scale)
    rest = 2.0 ** -20 * (score + 16)
    small = max(lens) * 2.0 ** -start * 112 * 0.125  # (the largest code is 112, the largest p is 1)
    tol = np.abs(want) * ((2.0 ** -8 + 2.0 ** -11 if dtype == "bf16" else 2.0 ** -23 + 2.0 ** -21) + rest[..., None]) + small
    err = np.abs(out.double().cpu().numpy().reshape(seqs, n, 4 * H, D) - want)
    assert np.all(err <= tol), f"worst {np.max(err / tol):.3g} of its tolerance, {np.max(err / np.abs(want)):.3g} of the result"
    assert np.all(np.abs(lse.double().cpu().numpy().reshape(seqs, n, 4 * H) - wl) <= rest)
    assert status() == 0


# ---------------------------------------------------------------- calls one after the other in one workspace

@pytest.mark.parametrize("dtype,n", [("bf16", 1), ("fp32", 2), ("bf16", 64)])
def test_calls_that_share_a_workspace(dtype, n):
    """The join starts beside the kernel whose partial results it reads: with other values in the same places before, each call's are its own."""
    rng, cache, table, lens, offs = setup(7 + n, [n], [9000], 64, "int8", 2, 128)
    args = dev(table), dev(lens), dev(offs)
    qs = [draw(rng, (n, 16, 128), dtype, w)[0] for w in (1.0, 3.0, 0.2, 5.0)]
    want = [cache.attention(q, *args, max_queries=n) for q in qs]
    workspace = torch.full((1 << 27,), 0x7F, dtype=torch.uint8, device=DEV)
    got = [cache.attention(qs[i % 4], *args, max_queries=n, workspace=workspace) for i in range(40)]
    for i, out in enumerate(got):
        assert torch.equal(out, want[i % 4]), i
    assert status() == 0


# ---------------------------------------------------------------- row tiles that end inside a warp

@pytest.mark.parametrize("fmt,D", [("int8", 128), ("e4m3", 64), ("e4m3", 128)])
@pytest.mark.parametrize("n,G", [(17, 1), (33, 1), (9, 5), (127, 1), (43, 3), (130, 1), (37, 7), (255, 1), (259, 1), (20, 13)])
def test_attention_row_tiles_that_end_inside_a_warp(n, G, fmt, D):
    """The prompt kernel with 1 to 255 rows in its last tile, whole items and split ones, and NaN in V that only some rows see."""
    news, befores = [n, n, 1], [0, 2000, 300]
    rng, cache, table, lens, offs = setup(n * G, news, befores, 16, fmt, 1, D)
    check_attention(cache, rng, "bf16", G, news, befores, table, lens, offs)
    if fmt == "e4m3":
        q, _ = draw(rng, (int(offs[-1]), G, D), "bf16")
        args = q, dev(table), dev(lens), dev(offs)
        clean = cache.attention(*args, max_queries=n)
        t, d = n - n // 3 - 1, D - 5  # a token of the first sequence, whose later queries see it
        page = cache.v_pages[int(table[0][t // 16])].view(torch.uint8)
        page[0, 0, d // 4, t % 16 // 4, d % 4, t % 4] = 0x7F
        out = cache.attention(*args, max_queries=n)
        want = torch.zeros_like(out, dtype=torch.bool)
        want[t:n, :, d] = True
        assert torch.equal(torch.isnan(out), want) and torch.equal(out[~want], clean[~want])
    assert status() == 0


# ---------------------------------------------------------------- waits that run out

@pytest.mark.parametrize("fmt,dtype,n,before,D", [
    ("int8", "bf16", 1, 900, 128), ("e4m3", "fp32", 3, 3000, 64),                               # the kernel for few queries
    ("int8", "bf16", 60, 100, 128), ("e4m3", "bf16", 300, 5000, 64), ("int8", "bf16", 17, 40000, 128),  # and for prompts
])
def test_waits_that_run_out_are_reported_and_the_next_call_is_right(fmt, dtype, n, before, D):
    """With an arrival fewer than its waits expect, a call ends by itself after their limit and says so; nothing outside its
    outputs is written, and the same call after it gives the same bits as before."""
    from adapter_gemm_linear_gb300 import arm_test_wait_timeout, device_status
    rng, cache, table, lens, offs = setup(n + D, [n, 2], [before, 70], 32, fmt, 2, D)
    T = int(offs[-1])
    q, _ = draw(rng, (T, 8, D), dtype)
    args = dev(table), dev(lens), dev(offs)
    want = cache.attention(q, *args, max_queries=n + 1, return_lse=True)
    held = [t.clone() for t in (cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales, q)]
    out = torch.full((T + 8, 8, D), 7.0, dtype=q.dtype, device=DEV)
    status()
    for limit in (5_000_000, 20_000_000):
        arm_test_wait_timeout(limit)
        cache.attention(q, *args, max_queries=n + 1, out=out[4:T + 4])
        st, site = device_status()
        assert st == 10 and 40 <= site <= 91, (st, site)
        assert bool((out[:4] == 7).all()) and bool((out[T + 4:] == 7).all())
        for t, h in zip((cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales, q), held):
            assert torch.equal(t.view(torch.uint8), h.view(torch.uint8))
        again = cache.attention(q, *args, max_queries=n + 1, return_lse=True)
        assert status() == 0
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


# ---------------------------------------------------------------- the binding

def test_a_workspace_that_the_kernels_cannot_use_is_refused():
    cache = KvCache(4, 2, 128, 16, "int8")
    tb, ln = torch.zeros((2, 2), dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    q = torch.zeros((2, 2, 128), device=DEV)
    for bad in (torch.empty(1 << 27, dtype=torch.uint8), torch.empty((1 << 27, 2), dtype=torch.uint8, device=DEV)[:, 0]):
        with pytest.raises(ValueError):
            cache.attention(q, tb, ln, workspace=bad)
    assert bool((cache.attention(q, tb, ln, workspace=torch.empty(1 << 25, device=DEV)) == 0).all())
    assert status() == 0


# ---------------------------------------------------------------- rotary positions out of range

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("axes,interleaved,rows", [(1, False, 4), (3, True, 4), (2, False, 4000)])
def test_pairs_of_positions_out_of_range_stay_as_they_are(dtype, axes, interleaved, rows):
    """To the bit, infinities, NaN and -0 among them; the other pairs of the row are turned as ever."""
    from adapter_gemm_linear_gb300 import device_status, rope, rope_tables
    rng = np.random.default_rng(axes)
    q, _ = draw(rng, (rows, 5, 64), dtype)
    q[1, :, ::3], q[1, :, 1::3], q[1, 2] = float("nan"), float("inf"), -0.0
    cos, sin = rope_tables(50, 64, device=DEV)
    pos = rng.integers(0, 50, (axes, rows)).astype(np.int32)
    ax = [int(a) for a in rng.integers(0, axes, 32)]
    good, _ = rope(q, None, cos, sin, dev(pos), axes=ax, interleaved=interleaved)
    pos[axes - 1, 1:] = 50
    pos[axes - 1, 2:] = -3
    status()
    out, _ = rope(q, None, cos, sin, dev(pos), axes=ax, interleaved=interleaved)
    st, row = device_status()
    assert st == 11 and 1 <= row < rows
    pairs = torch.tensor(ax) == axes - 1
    stays = (pairs.repeat_interleave(2) if interleaved else pairs.repeat(2)).to(DEV)
    bits = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(out.view(bits)[1:, :, stays], q.view(bits)[1:, :, stays])
    assert torch.equal(out.view(bits)[1:, :, ~stays], good.view(bits)[1:, :, ~stays])
    assert torch.equal(out.view(bits)[0], good.view(bits)[0])


def test_a_cache_keeps_no_growing_record_of_its_calls():
    """A server's calls have ever new numbers of rows: what the handle remembers of them stays bounded."""
    cache = KvCache(4, 1, 64, 16, "int8")
    tb, ln = torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    q = torch.zeros((700, 1, 64), device=DEV)
    for rows in range(1, 701):
        offs = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
        cache.attention(q[:rows], tb, ln, offs, max_queries=1)
    held = sum(len(x) for x in vars(cache).values() if isinstance(x, (dict, list, set)))
    assert held <= 256 and status() == 0


# ---------------------------------------------------------------- int8 pages filled token by token

def slowly(kind, tokens, D, rng):
    x = rng.normal(size=(tokens, 1, D))
    if kind == "growing":  # magnitudes 0.5% larger every token
        x = np.broadcast_to(x[:1], x.shape) * 1.005 ** np.arange(tokens)[:, None, None]
    elif kind == "turning":  # a large channel that turns slowly, as a low-frequency rotary pair does
        x[:, 0, 5] = 20 * np.cos(0.01 * np.arange(tokens) - 1.28)
    elif kind == "jumping":
        x = x * np.exp2(rng.integers(-60, 60, tokens))[:, None, None]
    return x


@pytest.mark.parametrize("kind", ["normal", "growing", "turning", "jumping"])
@pytest.mark.parametrize("dtype,D,page", [("bf16", 128, 128), ("fp32", 64, 32), ("bf16", 64, 16)])
def test_doubling_keeps_a_page_filled_token_by_token_within_a_step(kind, dtype, D, page):
    """Off by less than a step of the page's scale, which is less than twice the least one; and to the bit the definition's codes."""
    rng = np.random.default_rng(D + page)
    tokens = page + page // 2
    x = torch.from_numpy(slowly(kind, tokens, D, rng).astype(np.float32)).to(DT[dtype])
    cache = KvCache(2, 1, D, page, "int8", growth="doubling")
    table = dev(np.array([[1, 0]], np.int32))
    codes, scales = np.zeros((2, page, D), np.float32), np.zeros(2, np.float32)
    for t in range(tokens):
        row = x[t:t + 1].to(DEV)
        cache.append(row, row, table, dev(np.array([t + 1], np.int32)))
        p, i, v = t // page, t % page, x[t, 0].float().numpy()
        least = max(np.float32(np.abs(v).max()) / np.float32(127), np.float32(2.0 ** -120))
        s = scales[p]
        if i == 0:
            s = least
        while s < least:
            s = np.float32(2 * s)
        codes[p, :i] = np.rint(codes[p, :i] * np.float32(scales[p] / s)) if i else codes[p, :i]
        codes[p, i] = np.clip(np.rint(v / s), -127, 127)
        scales[p] = s
    assert np.array_equal(cache.k_scales.cpu().numpy()[[1, 0], 0], scales) and torch.equal(cache.k_scales, cache.v_scales)
    assert np.array_equal(R.unpack_k(cache.k_pages)[[1, 0], 0], codes) and np.array_equal(R.unpack_v(cache.v_pages)[[1, 0], 0], codes)
    got = cache.gather(table, dev(np.array([tokens], np.int32)), dev(np.array([0, tokens], np.int32)), rows=tokens, dtype=torch.float32)
    want = x.double().numpy()[:, 0]
    for y in got:
        err = np.abs(y.double().cpu().numpy()[:, 0] - want)
        for p in range(2):
            here = slice(p * page, min(tokens, (p + 1) * page))
            assert np.all(err[here] <= float(scales[p]) * (1 + 2.0 ** -20))
            assert float(scales[p]) < 2 * np.abs(want[here]).max() / 127 * (1 + 2.0 ** -22)
    assert status() == 0


@pytest.mark.parametrize("kind", ["normal", "growing", "turning"])
def test_the_least_scale_is_off_by_half_a_step_for_each_growth(kind):
    """The bound that the header gives for the default: (growths + 1) / 2 steps."""
    rng = np.random.default_rng(7)
    x = slowly(kind, 64, 64, rng).astype(np.float32)
    cache = KvCache(1, 1, 64, 64, "int8")
    table, growths, last = dev(np.zeros((1, 1), np.int32)), 0, 0.0
    for t in range(64):
        row = torch.from_numpy(x[t:t + 1]).to(DEV)
        cache.append(row, row, table, dev(np.array([t + 1], np.int32)))
        s = float(cache.k_scales[0, 0])
        growths += t > 0 and s > last
        last = s
    k, _ = cache.gather(table, dev(np.array([64], np.int32)), dev(np.array([0, 64], np.int32)), rows=64, dtype=torch.float32)
    assert float((k.cpu().double() - torch.from_numpy(x).double()).abs().max()) <= last * (growths + 1) / 2 * (1 + 2.0 ** -20)


def test_doubling_changes_nothing_where_no_scale_grows():
    """Whole pages at once, and e4m3: the same codes and scales with either growth."""
    for fmt, steps in (("int8", [96]), ("e4m3", [1] * 20 + [30, 46])):
        rng = np.random.default_rng(3)
        x, _ = draw(rng, (96, 2, 128), "bf16", 4.0)
        a, b = (KvCache(3, 2, 128, 32, fmt, growth=g) for g in ("least", "doubling"))
        table = dev(np.array([[2, 0, 1]], np.int32))
        for cache in (a, b):
            at = 0
            for n in steps:
                cache.append(x[at:at + n], x[at:at + n], table, dev(np.array([at + n], np.int32)), dev(np.array([0, n], np.int32)))
                at += n
        for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
            assert torch.equal(getattr(a, name).view(torch.uint8), getattr(b, name).view(torch.uint8))


@pytest.mark.parametrize("where", ["last page", "last page and least", "first page, out of the window"])
@pytest.mark.parametrize("huge", [40.0, 100.0, 119.0])
@pytest.mark.parametrize("dtype,fmt,n,before,page,D", [
    ("bf16", "int8", 5, 3000, 16, 128), ("fp32", "e4m3", 40, 300, 32, 64), ("bf16", "e4m3", 20, 20, 16, 64),
    ("bf16", "int8", 100, 700, 16, 128), ("bf16", "e4m3", 300, 4000, 32, 64), ("bf16", "int8", 150, 0, 16, 64),
])
def test_rows_are_untouched_by_scales_they_do_not_see(where, huge, dtype, fmt, n, before, page, D):
    """A later token's V, or one before the window, however large: each row's tolerance is by the V that it sees."""
    rng, cache, table, lens, offs = setup(before + n + page, [n], [before], page, fmt, 2, D)
    L, G, window = before + n, 4, 0
    pages = [int(p) for p in table[0] if p >= 0]
    if where.startswith("last"):
        cache.v_scales[pages[-1]] = float(2.0 ** huge)
        if where.endswith("least"):
            cache.v_scales[pages[:-1]] *= 2.0 ** -110
    else:
        cache.v_scales[pages[0]] = float(2.0 ** huge)
        window = L - page - n // 2  # the later rows do not see the first page
        if window < 1:
            window = 7
    ref = R.Paged(cache)
    q, qd = draw(rng, (n, 2 * G, D), dtype, 1.5)
    out, lse = cache.attention(q, dev(table), dev(lens), dev(offs), window=window, return_lse=True, max_queries=n)
    scale = np.float32(D ** -0.5).astype(np.float64)
    want, wl, spread, score = R.attention(ref, qd, table, lens, offs, scale, True, window)
    top = np.abs(ref.v).max((2, 3)) * ref.vs.astype(np.float64)  # of page and head
    vmax = np.zeros((n, 2 * G))
    for i in range(n):
        pos = before + i
        seen = pages[(max(0, pos - window + 1) if window else 0) // page:pos // page + 1]
        vmax[i] = np.repeat(top[seen].max(0), G)
    tol, ltol = bounds(dtype, want, wl, spread, score, L, vmax)
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= tol), f"worst {np.nanmax(err / tol):.3g} of its tolerance"
    assert np.all(np.abs(lse.double().cpu().numpy() - wl) <= ltol)
    assert status() == 0
