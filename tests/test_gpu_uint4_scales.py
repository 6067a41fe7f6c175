"""GPU tests of attention over the 4-bit cache where scales are far apart.

What the kernel for few queries promises beyond the bounds at the head of test_gpu_uint4_attention.py: with P the row's
largest p_j s_j / l (s_j token j's scale of V), each of the n terms p_j s_j code / l is off by at most 2^-33 P 15 (bf16) or
2^-44 P 15 (fp32) more than its 11 or 22 bits.  So, with A = sum p |s code| / l (no least values here), S = scale * sum |q k|:
    bf16: 2^-8 |o| + A (2^-11 + 2^-20 (S + 16)) + n 2^-33 15 P;  fp32: 2^-23 |o| + A (2^-21 + 2^-20 (S + 16)) + n 2^-44 15 P.
In fp32 calls a value s code + m enters as s (code - 8) and m + 8 s, whose products with p are rounded each for itself: of each
22 and 24 bits, so A is the sum over j of p_j (|s (code - 8)| + |m + 8 s|) / l there.  (With code = m = 0 that is 16 s and
not 0: a value of 0 that keeps 2^-21 of 16 s.  The kinds "at 0" have code = 8 and m = -8 s in that place, parts of 0 both.)
"""

import numpy as np
import pytest
import torch

import uint4_reference as U
from adapter_gemm_linear_gb300 import KvCache
from test_gpu_attention import DT, dev, status

pytestmark = pytest.mark.gpu

DEV = "cuda"
BLOCK = 224  # tokens: a step of 32 for each of a CTA's warps, which are seven at most


def kinds(kind, bits):
    """Per token: score in log2 (of a query of ones), V's scale, V's code (None: any), V's least value; `bits` below the row's
    largest p s the tail lies."""
    if kind.endswith(" at 0"):
        score, scale, code, _ = kinds(kind[:-5], bits)
        code = np.array([8 if c == 0 else c for c in code], object)
        return score, scale, code, np.where(code == 8, -8.0 * scale.astype(float), 0.0)
    low = bits + 0.75
    if kind == "ramp":  # each block just under and then just past the scores that the row's maximum is held for
        score = [0.0, 8 - 2.0 ** -7, 16.25]
        scale, code = [1.5] * 3, [0] * 3
        tail = score[-1] - low, 1.5, 15
    elif kind == "creep":  # (of the query of ones; one of nines grows past it in every block)
        score = [float(i) for i in range(8)]
        scale, code = [1.5 * 4.0 ** -i for i in range(8)], [0] * 8
        tail = -low, 1.5, 15
    else:  # a first block with large V that loses its weight
        score, code = [0.0], [15]
        scale = [{"lost 1e-4": 2000.0, "lost 2^-13": 4096.0, "lost 2^-20": 4000.0, "lost 2^-24": 4096.0}[kind]]
        tail = None, {"lost 1e-4": 1e-4, "lost 2^-13": 2.0 ** -13, "lost 2^-20": 2.0 ** -20, "lost 2^-24": 2.0 ** -24}[kind], None
    parts = [np.repeat(np.array(x, object), BLOCK) for x in (score, scale, code)]
    ends = [np.array([t] * 640, object) for t in tail]
    if tail[0] is None:
        ends[0] = 60 - np.arange(640) % 61 / 30.0
    return [np.concatenate(x) for x in zip(parts, ends)] + [np.zeros(len(parts[0]) + 640)]


@pytest.mark.parametrize("kind", ["ramp", "creep", "ramp at 0", "creep at 0", "lost 1e-4", "lost 2^-13", "lost 2^-20", "lost 2^-24"])
@pytest.mark.parametrize("dtype,D,G,n", [("bf16", 128, 2, 1), ("bf16", 64, 8, 1), ("bf16", 128, 16, 1), ("bf16", 64, 4, 4), ("fp32", 128, 2, 1),
                                         ("fp32", 64, 8, 2)])
def test_large_scales_that_lose_their_weight(kind, dtype, D, G, n):
    rng = np.random.default_rng(D + G + n)
    S, H, page = 64, 8, 16  # (all sequences have the same tokens: CTAs have items' beginnings with long parts of their rest)
    score, vs, code, least = kinds(kind, 25 if dtype == "bf16" else 36)
    L = len(score)
    score, vs = score.astype(np.float16).astype(np.float64), vs.astype(np.float16).astype(np.float64)
    pages = (L + page - 1) // page
    cache = KvCache(pages, H, D, page, "uint4", device=DEV)
    codes = np.zeros((pages * page, D), int)
    codes[:L] = [[c] * D if c is not None else rng.integers(0, 16, D) for c in code]
    byte, high = U.places(D)["v"]
    v = np.zeros((pages, D // 64 * 512), np.uint8)
    for p in range(pages):
        np.add.at(v[p], byte.reshape(-1), (codes[p * page:(p + 1) * page] << (4 * high)).astype(np.uint8).reshape(-1))
    cache.v_pages.view(pages, H, -1).copy_(torch.from_numpy(v)[:, None])
    for t, x, place in ((cache.k_scales, score, 1), (cache.v_scales, vs, 0), (cache.v_scales, least, 1)):
        y = np.zeros((pages * page,), np.float16)
        y[:L] = x
        t[..., place] = torch.from_numpy(y.reshape(pages, 1, 1, 1, page)).to(DEV)
    heads = np.where(np.arange(H * G) % 2 == 0, 1.0, 9.0 if kind == "creep" else 1.0)
    q = torch.from_numpy(np.tile(heads[None, :, None], (S * n, 1, D))).to(DT[dtype]).to(DEV)
    sm = np.float32(np.log(2.0) / D)
    table = dev(np.tile(np.arange(pages, dtype=np.int32), (S, 1)))
    lens, offs = dev(np.full(S, L, np.int32)), dev(np.arange(0, S * n + 1, n, dtype=np.int32))
    out, lse = cache.attention(q, table, lens, offs, max_queries=n, scale=float(sm), return_lse=True)
    assert status() == 0
    out, lse = out.double().cpu().numpy().reshape(S, n, H * G, D), lse.double().cpu().numpy().reshape(S, n, H * G)
    for i in range(n):
        for h, size in enumerate(heads[:2]):
            seen = L - n + 1 + i
            z = score[:seen] * size * D * np.float64(sm)
            p = np.exp(z - z.max())
            p /= p.sum()
            ps, pm = p * vs[:seen], p @ least[:seen]
            want = ps @ codes[:seen] + pm
            if dtype == "bf16":
                size_of = ps @ codes[:seen] + p @ np.abs(least[:seen])
            else:
                size_of = ps @ np.abs(codes[:seen] - 8) + p @ np.abs(least[:seen] + 8 * vs[:seen])
            most = np.abs(score[:seen]).max() * size * D * np.float64(sm)
            bits, step = (2.0 ** -8, 2.0 ** -33) if dtype == "bf16" else (2.0 ** -23, 2.0 ** -44)
            tol = np.abs(want) * bits + size_of * ((2.0 ** -11 if dtype == "bf16" else 2.0 ** -21) + 2.0 ** -20 * (most + 16)) + \
                seen * step * 15 * ps.max()
            err = np.abs(out[:, i, h::2] - want)
            assert np.all(err <= tol), f"{np.max(err / np.maximum(tol, 1e-300)):.3g} of its tolerance, {np.max(err / np.maximum(np.abs(want), 1e-300)):.3g} of the result"
            want = z.max() + np.log(np.exp(z - z.max()).sum())
            assert np.all(np.abs(lse[:, i, h::2] - want) <= 2.0 ** -20 * (most + 16))
