"""GPU tests: what a query does not see of the 4-bit cache does not reach its result, whatever it is."""

import numpy as np
import pytest
import torch

import uint4_reference as U
from adapter_gemm_linear_gb300 import KvCache  # noqa: F401
from test_gpu_attention import bounds, dev, draw, status
from test_gpu_uint4_attention import many_queries, setup

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def run(cache, q, table, lens, offs, most, causal, window, with_lse):
    r = cache.attention(q, dev(table), dev(lens), dev(offs), max_queries=most, causal=causal, window=window, return_lse=with_lse)
    assert status() == 0
    out, lse = r if with_lse else (r, None)
    return out.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()


def compare(cache, ref, q, qd, table, lens, offs, most, window, dtype, G, hidden=None):
    """Of all results but the `hidden` ones [rows, dimensions], which are not finite: right, with lse and without."""
    T, Hq, D = qd.shape
    many = many_queries(dtype, T, cache, G, table, most)
    for with_lse in (True, False):
        out, lse = run(cache, q, table, lens, offs, most, True, window, with_lse)
        rounded = "" if not many else "v" if with_lse else "kv"
        want, wl, spread, score, vmax = U.attention(ref, qd, table, lens, offs, np.float32(D ** -0.5).astype(np.float64), True, window, rounded)
        tol, ltol = bounds(dtype, want, wl, spread, score, max(lens), vmax)
        keep = np.ones((T, D), bool) if hidden is None else ~hidden
        keep = np.broadcast_to(keep[:, None], want.shape)
        assert np.all(np.abs(out - want)[keep] <= tol[keep]), np.argwhere(~(np.abs(out - want) <= tol) & keep)[:5]
        assert not np.any(np.isfinite(out[~keep]))
        if lse is not None:
            assert np.all(np.abs(lse - wl) <= ltol)


CALLS = [("bf16", [4, 3], [100, 61], 2, 128), ("bf16", [16, 9], [100, 500], 8, 128), ("bf16", [7, 9], [300, 20], 4, 64), ("fp32", [5, 8], [40, 90], 4, 128),
         ("fp32", [30, 8], [40, 900], 1, 64), ("bf16", [300, 40], [500, 2000], 4, 128), ("bf16", [200, 250], [3000, 60], 8, 64)]


@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("value", [(NAN, 0.5), (0.5, NAN), (INF, 0.5), (0.5, -INF)])
@pytest.mark.parametrize("dtype,news,befores,G,D", CALLS)
def test_tokens_that_some_rows_see(dtype, news, befores, G, D, value, window):
    """A scale or least value of V that is no number reaches the rows that see its token, in its 64 dimensions, and no others."""
    H = 2
    rng, cache, table, lens, offs = setup(news[0] + D, news, befores, 16, H, D)
    q, qd = draw(rng, (int(offs[-1]), H * G, D), dtype)
    ref = U.Paged4(cache)
    hidden = np.zeros((int(offs[-1]), D), bool)
    for s in range(2):
        at, h = int(lens[s]) - (news[s] + 1) // 2, s % (D // 64)
        cache.v_scales[int(table[s][at // 16]), :, 0, h, at % 16] = torch.tensor(value, dtype=torch.float16, device="cuda")
        pos = np.arange(lens[s] - news[s], lens[s])
        seen = (at <= pos) & ((at > pos - window) if window else True)
        assert seen.any() and not seen.all()
        hidden[offs[s]:offs[s + 1], 64 * h:64 * h + 64] |= seen[:, None]
    compare(cache, ref, q, qd, table, lens, offs, max(news), window, dtype, G, hidden)


@pytest.mark.parametrize("value", [(NAN, NAN), (INF, -INF), (60000.0, 60000.0)])
@pytest.mark.parametrize("window", [20, 77])
@pytest.mark.parametrize("dtype,news,befores,G,D", CALLS + [("bf16", [1, 1], [100, 333], 8, 128), ("fp32", [1, 1], [100, 333], 2, 64)])
def test_tokens_before_the_window_that_were_never_written(dtype, news, befores, G, D, window, value):
    H = 2
    rng, cache, table, lens, offs = setup(news[0] + D, news, befores, 16, H, D)
    q, qd = draw(rng, (int(offs[-1]), H * G, D), dtype)
    ref = U.Paged4(cache)
    for s in range(2):
        for at in range(max(0, befores[s] - window + 1)):
            for t in (cache.k_scales, cache.v_scales):
                t[int(table[s][at // 16]), :, 0, :, at % 16] = torch.tensor(value, dtype=torch.float16, device="cuda")
    compare(cache, ref, q, qd, table, lens, offs, max(news), window, dtype, G)


@pytest.mark.parametrize("value", [(NAN, 0.5), (0.5, NAN), (INF, 0.5), (0.5, -INF)])
@pytest.mark.parametrize("dtype,news,befores,G,D", [c for c in CALLS if c[-1] == 128] + [("bf16", [1, 1], [100, 333], 8, 128)])
def test_tokens_that_all_rows_see(dtype, news, befores, G, D, value):
    """The other 64 dimensions are right."""
    H = 2
    rng, cache, table, lens, offs = setup(news[0] + D + 1, news, befores, 16, H, D)
    q, qd = draw(rng, (int(offs[-1]), H * G, D), dtype)
    ref = U.Paged4(cache)
    hidden = np.zeros((int(offs[-1]), D), bool)
    for s in range(2):
        cache.v_scales[int(table[s][0]), :, 0, s, 5] = torch.tensor(value, dtype=torch.float16, device="cuda")
        hidden[offs[s]:offs[s + 1], 64 * s:64 * s + 64] = True
    compare(cache, ref, q, qd, table, lens, offs, max(news), 0, dtype, G, hidden)
