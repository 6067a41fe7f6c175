"""GPU tests: with a window, table entries of pages that no query of the call sees are not needed and may name no page."""

import numpy as np
import pytest

import attention_reference as R
import uint4_reference as U
from adapter_gemm_linear_gb300 import KvCache
from test_gpu_attention import bounds, dev, draw, status
from test_gpu_uint4_attention import many_queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int8", "e4m3", "uint4"])
@pytest.mark.parametrize("dtype,news,befores,G,window,page", [
    ("bf16", [1, 1], [100, 333], 8, 20, 16), ("fp32", [4, 3], [100, 333], 2, 33, 16), ("bf16", [9, 16], [200, 700], 4, 50, 16),
    ("bf16", [300, 200], [1000, 1100], 4, 77, 16), ("bf16", [300, 200], [1000, 1100], 8, 20, 32), ("bf16", [600, 40], [2000, 5000], 2, 130, 64),
])
def test_pages_before_the_window(fmt, dtype, news, befores, G, window, page):
    H, D = 2, 128
    rng = np.random.default_rng(sum(news) + window)
    table, lens, offs, num = R.make_batch(rng, news, befores, page)
    cache = KvCache(num, H, D, page, fmt, device="cuda")
    (U.random_cache if fmt == "uint4" else R.random_codes)(rng, cache)
    q, qd = draw(rng, (int(offs[-1]), H * G, D), dtype)
    sm = np.float32(D ** -0.5).astype(np.float64)
    if fmt == "uint4":
        rounded = "v" if many_queries(dtype, int(offs[-1]), cache, G, table, max(news)) else ""
        want, wl, spread, score, vmax = U.attention(U.Paged4(cache), qd, table, lens, offs, sm, True, window, rounded)
    else:
        ref = R.Paged(cache)
        want, wl, spread, score = R.attention(ref, qd, table, lens, offs, sm, True, window)
        vmax = np.max(np.abs(ref.v) * ref.vs[:, :, None, None])
    tol, ltol = bounds(dtype, want, wl, spread, score, max(lens), vmax)
    for _ in range(2):
        out, lse = cache.attention(q, dev(table), dev(lens), dev(offs), max_queries=max(news), window=window, return_lse=True)
        assert status() == 0
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol) and np.all(np.abs(lse.double().cpu().numpy() - wl) <= ltol)
        for s in range(2):
            table[s, :max(0, befores[s] - window + 1) // page] = (-1, num)[s]
