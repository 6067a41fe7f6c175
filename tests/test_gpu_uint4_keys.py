"""GPU tests of attention over the 4-bit cache: keys whose scales are as large as the format has them, and keys far from 0."""

import numpy as np
import pytest
import torch

from test_gpu_uint4_attention import check, setup

pytestmark = pytest.mark.gpu

CALLS = [("bf16", 1, 300), ("fp32", 3, 200), ("bf16", 200, 1900), ("bf16", 70, 900)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,n,before", CALLS)
def test_the_largest_scales(dtype, n, before, D):
    """All 16 values within f16's range: scales past 8192 with least values near the range's lower end."""
    rng, cache, table, lens, offs = setup(n + D, [n, 2], [before, 40], 16, 2, D, room=2048)
    sc = np.empty(tuple(cache.k_scales.shape), np.float64)
    sc[..., 0] = rng.uniform(8100, 8700, sc.shape[:-1])
    sc[..., 1] = -7.5 * sc[..., 0] + rng.uniform(-200, 200, sc.shape[:-1])
    cache.k_scales.copy_(torch.from_numpy(sc.astype(np.float16)))
    sc = cache.k_scales.double()
    assert float((sc[..., 0] * 15 + sc[..., 1]).max()) < 65504 and float(sc[..., 1].min()) > -65504
    check(cache, rng, dtype, 8, [n, 2], table, lens, offs, q_width=1e-3, scale=0.02)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,n,before", CALLS)
def test_keys_far_from_zero(dtype, n, before, D):
    rng, cache, table, lens, offs = setup(n + D + 1, [n, 2], [before, 40], 16, 2, D, room=2048)
    sc = np.empty(tuple(cache.k_scales.shape), np.float64)
    sc[..., 0] = 0.3 * np.exp(0.3 * rng.normal(size=sc.shape[:-1]))
    sc[..., 1] = 100 + rng.normal(size=sc.shape[:-1])
    cache.k_scales.copy_(torch.from_numpy(sc.astype(np.float16)))
    check(cache, rng, dtype, 8, [n, 2], table, lens, offs)
