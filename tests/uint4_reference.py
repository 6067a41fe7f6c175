"""Plain restatements of the 4-bit cache on the CPU, apart from the library, reading the documented layout index by index."""

from __future__ import annotations

import numpy as np
import torch


def places(D):
    """Of (token, dimension) of a tile: byte and nibble in K's pages, and in V's."""
    out = {}
    for name in ("k", "v"):
        byte, high = np.empty((16, D), int), np.empty((16, D), int)
        for t in range(16):
            for d in range(D):
                r = d % 64
                if name == "k":
                    g = next(g for g in range(8) if t in (4 * (g // 2) + g % 2, 4 * (g // 2) + g % 2 + 2))
                    second = t - (4 * (g // 2) + g % 2)
                    pair = [(0, 2), (4, 6), (1, 3), (5, 7)]
                    i = next(i for i in range(4) if r % 8 in pair[i])
                    at, hi = 16 * (4 * g + r // 16) + 8 * (second // 2) + 4 * (r % 16 // 8) + i, pair[i].index(r % 8)
                else:
                    g = r % 32 // 4
                    j = next(j for j in range(4) if r - 4 * g - 32 * (j // 2) - 2 * (j % 2) in (0, 1))
                    hi = r - 4 * g - 32 * (j // 2) - 2 * (j % 2)
                    at = 16 * (4 * g + t // 4) + 4 * j + [0, 2, 1, 3].index(t % 4)
                byte[t, d], high[t, d] = d // 64 * 512 + at, hi
        assert len(set(zip(byte.flat, high.flat))) == 16 * D
        out[name] = byte, high
    return out


class Paged4:
    """Codes int [pages, heads, page, D], scales and least values float64 [pages, heads, page, D/64]; attention_reference's
    tokens() and attention() read it by way of `values`."""

    def __init__(self, cache):
        self.P, self.D, self.H = cache.page_tokens, cache.head_dim, cache.num_heads
        self.where = places(self.D)
        for name in ("k", "v"):
            setattr(self, name, self.unpack(getattr(cache, name + "_pages"), name))
            setattr(self, name + "s", self.scales(getattr(cache, name + "_scales")))

    def unpack(self, pages, name):
        byte, high = self.where[name]
        x = pages.cpu().numpy()
        x = x.reshape(x.shape[0], x.shape[1], self.P // 16, -1)[..., byte]  # [.., 16, D]
        return ((x >> (4 * high)) & 15).reshape(x.shape[0], x.shape[1], self.P, self.D).astype(int)

    def scales(self, s):
        s = s.cpu().numpy().astype(np.float16)  # [pages, heads, tiles, D/64, 16, 2]
        return s.transpose(0, 1, 2, 4, 3, 5).reshape(s.shape[0], s.shape[1], self.P, self.D // 64, 2)

    def values(self, name):
        """float64 [pages, heads, page, D]"""
        s = getattr(self, name + "s").astype(np.float64).repeat(64, axis=3)
        with np.errstate(invalid="ignore"):
            return getattr(self, name) * s[..., 0] + s[..., 1]


def quantise(x):
    """fp32 [..., 64] -> codes, (scale, least) in f16: the definition's fp32 steps."""
    x = np.where(np.isnan(x), np.float32(0), x.astype(np.float32))
    fin = np.isfinite(x)
    x = np.where(fin, np.clip(x, np.float32(-2.0 ** 15), np.float32(2.0 ** 15)), x)
    lo = np.where(fin, x, np.float32(np.inf)).min(-1)
    hi = np.where(fin, x, np.float32(-np.inf)).max(-1)
    none = ~fin.any(-1)
    lo, hi = np.where(none, np.float32(0), lo), np.where(none, np.float32(0), hi)
    m = lo.astype(np.float16)
    s = ((hi - lo) * np.float32(1 / 15)).astype(np.float16)
    s32, m32 = s.astype(np.float32)[..., None], m.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((x - m32) / s32)
    code = np.where(s32 > 0, np.clip(np.nan_to_num(q, posinf=15, neginf=0), 0, 15), 0).astype(int)
    return code, np.stack((s, m), -1)


def append(ref: Paged4, x, which, table, lens, offs):
    """x: float64 [rows, H, D] (values of the call's dtype)."""
    codes, scales = getattr(ref, which), getattr(ref, which + "s")
    for s in range(len(lens)):
        n, L = offs[s + 1] - offs[s], lens[s]
        for i in range(n if L else 0):
            pos = L - n + i
            page = table[s][pos // ref.P]
            c, sc = quantise(x[offs[s] + i].reshape(ref.H, ref.D // 64, 64))
            codes[page, :, pos % ref.P] = c.reshape(ref.H, ref.D)
            scales[page, :, pos % ref.P] = sc


class Values:
    """What attention_reference.attention reads: `k`, `v` with scales of 1."""

    def __init__(self, ref: Paged4):
        self.P, self.D, self.H = ref.P, ref.D, ref.H
        self.k, self.v = ref.values("k"), ref.values("v")
        self.ks = self.vs = np.ones(self.k.shape[:2], np.float32)


def random_cache(rng, cache, spread=0.3, size=1.0):
    """Any codes, and scales as normal values have them, tokens of varying magnitude; some with scale 0."""
    for t in (cache.k_pages, cache.v_pages):
        t.view(-1).copy_(torch.from_numpy(rng.integers(0, 256, t.numel(), dtype=np.uint8)))
    for t in (cache.k_scales, cache.v_scales):
        z = np.exp(spread * rng.normal(size=t.shape[:-1])) * size
        s = np.stack((0.3 * z, z * (-2.3 + 0.4 * rng.normal(size=z.shape))), -1)
        s[..., 0][rng.random(z.shape) < 0.02] = 0
        t.copy_(torch.from_numpy(s.astype(np.float16)))


def attention(ref: Paged4, q, table, lens, offs, scale, causal=True, window=0, rounded=""):
    """q: float64 [rows, Hq, D] -> (out, lse, spread, score, vmax): the exact result, and per row and head what error
    bounds need: the largest over dimensions of sum p |v|, the largest of scale * sum |q k|, and the largest |v| that
    it sees.  In them |k| and |v| stand for |scale code| + |least|, the parts that the products take.  `rounded`: the
    values of those ("v", "kv") rounded to f16 first, and |k| and |v| theirs."""
    T, Hq, D = q.shape
    G = Hq // ref.H
    vals, mags = {}, {}
    for name in ("k", "v"):
        s = getattr(ref, name + "s").astype(np.float64).repeat(64, 3)
        with np.errstate(invalid="ignore"):
            parts = getattr(ref, name) * s[..., 0], s[..., 1]
            vals[name] = parts[0] + parts[1]
            mags[name] = np.abs(parts[0]) + np.abs(parts[1])
            if name in rounded:
                vals[name] = vals[name].astype(np.float16).astype(np.float64)
                mags[name] = np.abs(vals[name])
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    spread, score, vmax = np.zeros((T, Hq)), np.zeros((T, Hq)), np.zeros((T, Hq))
    for s in range(len(lens)):
        n, L = offs[s + 1] - offs[s], lens[s]
        if L == 0 or n == 0:
            continue

        def tokens(x):
            j = np.arange(L)
            return np.stack([x[table[s][i // ref.P], :, i % ref.P] if 0 <= table[s][i // ref.P] < x.shape[0] else
                             np.zeros((ref.H, D)) for i in j])

        k, v, km, vm = (tokens(x) for x in (vals["k"], vals["v"], mags["k"], mags["v"]))
        pos, j = np.arange(L - n, L)[:, None], np.arange(L)[None, :]
        ok = np.ones((n, L), bool) if not causal else j <= pos
        if window:
            ok = ok & (j > pos - window)
        rows = slice(offs[s], offs[s + 1])
        for h in range(Hq):
            qs, hk = q[rows, h], h // G
            z = np.where(ok, qs @ k[:, hk].T * scale, -np.inf)
            m = z.max(1, keepdims=True)
            p = np.exp(z - m)
            l = p.sum(1, keepdims=True)
            out[rows, h] = p @ v[:, hk] / l
            lse[rows, h] = (m + np.log(l))[:, 0]
            spread[rows, h] = (p @ vm[:, hk] / l).max(1)
            score[rows, h] = np.where(ok, np.abs(qs) @ km[:, hk].T * scale, 0.0).max(1)
            vmax[rows, h] = np.where(ok, vm[:, hk].max(1)[None], 0.0).max(1)
    return out, lse, spread, score, vmax
