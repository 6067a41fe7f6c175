"""GPU parity of the 4-bit cache's writing and reading (KvCache(fmt="uint4")) with plain restatements.

Codes and scales are equal, bit for bit (both sides do the definition's fp32 steps); a gathered value is one fp32
sum of an exact product, 2^-24 of |code scale| + |least| (an fp32 fma, or that again where the scale's power of two is taken
along: exact), in bf16 one more rounding, 2^-8 of the value."""

import numpy as np
import pytest
import torch

import attention_reference as R
import uint4_reference as U
from adapter_gemm_linear_gb300 import KvCache, device_status, kv_pages_bytes, kv_scales_bytes
from test_gpu_attention import BATCHES, DT, dev, draw, status
from test_gpu_attention_layouts import LAYOUTS, laid_out

pytestmark = pytest.mark.gpu

DEV = "cuda"


def make(rng, news, befores, page, D, H, fill=True):
    table, lens, offs, num = R.make_batch(rng, news, befores, page, room=3)
    cache = KvCache(num, H, D, page, "uint4", device=DEV)
    if fill:
        U.random_cache(rng, cache)
    return cache, U.Paged4(cache), table, lens, offs, (dev(table), dev(lens), dev(offs))


def check(cache, ref):
    got = U.Paged4(cache)
    for name in ("k", "v"):
        np.testing.assert_array_equal(getattr(got, name), getattr(ref, name))
        np.testing.assert_array_equal(getattr(got, name + "s").view(np.int16), getattr(ref, name + "s").view(np.int16))


def check_gather(ref, kv, table, lens, offs, dtype):
    for name, got in zip(("k", "v"), kv):
        v, s = ref.values(name), getattr(ref, name + "s").astype(np.float64).repeat(64, 3)
        mag = np.abs(getattr(ref, name) * s[..., 0]) + np.abs(s[..., 1])
        got = got.double().cpu().numpy()
        for q in range(len(lens)):
            for i in range(offs[q + 1] - offs[q] if lens[q] else 0):
                pos = lens[q] - (offs[q + 1] - offs[q]) + i
                page, t = table[q][pos // ref.P], pos % ref.P
                want = v[page, :, t]
                tol = 2.0 ** -24 * mag[page, :, t] + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
                assert np.all(np.abs(got[offs[q] + i] - want) <= tol), (name, q, pos)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,D,H", [("bf16", 128, 2), ("fp32", 64, 3), ("bf16", 64, 1), ("fp32", 128, 5)])
def test_append_and_gather(page, dtype, D, H):
    rng = np.random.default_rng(page + D)
    for news, befores in BATCHES:
        cache, ref, table, lens, offs, (tb, ln, of) = make(rng, news, befores, page, D, H)
        k, kd = draw(rng, (sum(news), H, D), dtype, 2.0, pad=16)
        v, vd = draw(rng, (sum(news), H, D), dtype, 0.01, pad=8)
        args = (tb, ln, of) if any(n != 1 for n in news) else (tb, ln)
        cache.append(k, v, *args)
        U.append(ref, kd, "k", table, lens, offs)
        U.append(ref, vd, "v", table, lens, offs)
        check(cache, ref)
        whole = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
        for out in ("bf16", "fp32"):
            kv = cache.gather(tb, ln, dev(whole), rows=int(whole[-1]), dtype=DT[out])
            check_gather(ref, kv, table, lens, whole, out)
            kv = cache.gather(*args, rows=sum(news), dtype=DT[out])
            check_gather(ref, kv, table, lens, offs, out)
    assert status() == 0


def test_a_sequence_written_in_any_pieces_is_the_same():
    rng = np.random.default_rng(3)
    L, H, D = 150, 2, 128
    k, v = draw(rng, (L, H, D), "bf16")[0], draw(rng, (L, H, D), "bf16")[0]
    whole = KvCache(5, H, D, 32, "uint4", device=DEV)
    table = dev(np.array([[3, 1, 4, 0, 2]], np.int32))
    whole.append(k, v, table, dev(np.array([L], np.int32)), dev(np.array([0, L], np.int32)))
    pieces = KvCache(5, H, D, 32, "uint4", device=DEV)
    at = 0
    while at < L:
        n = min(L - at, int(rng.integers(1, 9)))
        pieces.append(k[at:at + n], v[at:at + n], table, dev(np.array([at + n], np.int32)), dev(np.array([0, n], np.int32)))
        at += n
    for a, b in ((whole.k_pages, pieces.k_pages), (whole.v_pages, pieces.v_pages), (whole.k_scales, pieces.k_scales),
                 (whole.v_scales, pieces.v_scales)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_values_at_the_edges(dtype):
    """Zeros, constants, infinities, NaN, values too large, too small, and next to a half."""
    D, H = 64, 1
    rng = np.random.default_rng(1)
    rows = [np.zeros(64), np.full(64, 3.25), np.full(64, -1e30), np.full(64, np.inf), np.full(64, np.nan), np.full(64, -np.inf)]
    x = rng.normal(size=64)
    for where, what in ((3, np.inf), (4, -np.inf), (5, np.nan), (6, 1e30), (7, -4e4), (8, 1e-30), (9, -0.0)):
        y = x.copy()
        y[where] = what
        rows.append(y)
    rows.append(np.where(np.arange(64) % 2, np.inf, -np.inf))
    rows.append(np.where(np.arange(64) % 3 == 0, np.nan, np.inf))
    rows += [x * 2.0 ** e for e in (-40, -24, -20, -14, 10, 14, 20, 100)]
    rows.append(np.arange(64) / 8.0 + 2)  # (halves: 15 steps of 0.525)
    rows.append((np.arange(64) % 31) / 2.0)  # exact halves: ties go to even codes
    rows.append(-(np.arange(64) % 31) / 2.0 + 4096)
    x = torch.from_numpy(np.array(rows, np.float32)).to(DT[dtype])[:, None]
    n = len(rows)
    cache = KvCache(3, H, D, 32, "uint4", device=DEV)
    ref = U.Paged4(cache)
    table, lens, offs = np.array([[2, 0, 1]], np.int32), np.array([n], np.int32), np.array([0, n], np.int32)
    cache.append(x.to(DEV), x.flip(0).contiguous().to(DEV), dev(table), dev(lens), dev(offs))
    U.append(ref, x.double().numpy(), "k", table, lens, offs)
    U.append(ref, x.flip(0).double().numpy(), "v", table, lens, offs)
    check(cache, ref)
    k, v = cache.gather(dev(table), dev(lens), dev(offs), rows=n, dtype=torch.float32)
    assert bool(k.isfinite().all()) and bool(v.isfinite().all())
    # a value within the range is within half a step, and the scale's rounding, of its place
    fin = x.double().numpy()[:, 0]
    ok = np.isfinite(fin).all(1) & (np.abs(fin) <= 2.0 ** 15).all(1)
    err = np.abs(k.double().cpu().numpy()[:, 0] - fin)[ok]
    step = (fin.max(1) - fin.min(1))[ok] / 15
    # half a step of the f16 scale; the ends: 15 steps each off by 2^-11 (or 2^-25), and the least value's rounding
    tol = step * (0.5 + 16 * 2.0 ** -11) + 16 * 2.0 ** -25 + 2.0 ** -11 * np.abs(fin.min(1))[ok]
    assert np.all(err <= tol[:, None])


def test_bad_tables_lengths_and_offsets():
    rng = np.random.default_rng(2)
    H, D = 2, 64
    cache, ref, table, lens, offs, (tb, ln, of) = make(rng, [2, 2, 2, 2], [30, 0, 5, 40], 16, D, H)
    before = [t.clone() for t in (cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales)]
    k, kd = draw(rng, (8, H, D), "bf16")
    status()
    t2 = table.copy()
    t2[0, 1] = 1 << 20  # page of the new tokens
    t2[1, 0] = -1
    cache.append(k, k, dev(t2), ln, of)
    st, s = device_status()
    assert st == 11 and s in (0, 1)
    U.append(ref, kd[4:], "k", table[2:], lens[2:], offs[2:] - 4)
    U.append(ref, kd[4:], "v", table[2:], lens[2:], offs[2:] - 4)
    check(cache, ref)
    # reads of such pages are zeros
    kk, vv = cache.gather(dev(t2), ln, of, rows=8, dtype=torch.float32)
    assert device_status()[0] == 11
    assert bool((kk[:4] == 0).all()) and bool((vv[:4] == 0).all()) and bool((kk[4:] != 0).any())
    for t, b in zip((cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales), before):
        t.copy_(b)
    bad_lens = lens.copy()
    bad_lens[0], bad_lens[1], bad_lens[2], bad_lens[3] = -3, 1 << 30, 1, 0  # (the third has more rows than tokens)
    cache.append(k, k, tb, dev(bad_lens), of)
    assert device_status()[0] in (8, 11)
    out = torch.full((8, H, D), 7.0, device=DEV)
    cache.gather(tb, dev(bad_lens), of, k_out=out, v_out=torch.empty_like(out))
    assert device_status()[0] in (8, 11) and bool((out == 7).all())
    for t, b in zip((cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales), before):
        assert torch.equal(t, b)
    cache.append(k, k, tb, ln, dev(np.array([0, 5, 3, 6, 99], np.int32)))
    assert device_status()[0] == 8


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_layouts(layout, dtype):
    rng = np.random.default_rng(4)
    H, D, news, befores = 2, 128, [5, 40, 1], [3, 0, 20]
    cache, _, table, lens, offs, args = make(rng, news, befores, 16, D, H)
    other = KvCache(cache.num_pages, H, D, 16, "uint4", k_pages=cache.k_pages.clone(), v_pages=cache.v_pages.clone(),
                    k_scales=cache.k_scales.clone(), v_scales=cache.v_scales.clone())
    k, v = (draw(rng, (46, H, D), dtype)[0].contiguous() for _ in range(2))
    cache.append(k, v, *args)
    other.append(laid_out(k, layout)[0], laid_out(v, layout)[0], *args)
    for name in ("k_pages", "v_pages", "k_scales", "v_scales"):
        assert torch.equal(getattr(cache, name), getattr(other, name))
    want = cache.gather(*args, rows=46, dtype=DT[dtype])
    outs = [laid_out(torch.zeros_like(k), layout) for _ in range(2)]
    cache.gather(*args, k_out=outs[0][0], v_out=outs[1][0])
    for (view, whole, outside), w in zip(outs, want):
        assert torch.equal(view, w) and bool((whole[outside] == 7).all())


def test_bytes_and_buffers():
    cache = KvCache(7, 3, 128, 32, "uint4", device=DEV)
    assert cache.k_pages.nbytes == cache.v_pages.nbytes == kv_pages_bytes(7, 3, 128, 32, "uint4") == 7 * 3 * 128 * 32 // 2
    assert cache.k_scales.nbytes == cache.v_scales.nbytes == kv_scales_bytes(7, 3, 128, 32, "uint4") == 7 * 3 * 128 * 32 // 16
    with pytest.raises(ValueError):
        KvCache(7, 3, 128, 32, "uint4", k_pages=torch.zeros((7, 3, 2, 2, 16, 64), dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        KvCache(7, 3, 128, 32, "uint4", k_scales=torch.zeros((7, 3), device=DEV))
