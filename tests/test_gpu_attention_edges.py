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
