"""Plain float64 restatements of rotary positions, the 8-bit paged cache and
attention over it, on the CPU and apart from the library: loops over
sequences, pages and heads, reading the documented page layout index by index.
"""

from __future__ import annotations

import math

import numpy as np
import torch

MIN_SCALE = np.float32(2.0 ** -120)


class Paged:
    """A cache on the CPU: codes as float64 [pages, heads, page, D], NaN kept, and fp32 scales."""

    def __init__(self, cache):
        self.fmt, self.P, self.D, self.H = cache.fmt, cache.page_tokens, cache.head_dim, cache.num_heads
        self.k = unpack_k(cache.k_pages)
        self.v = unpack_v(cache.v_pages)
        self.ks = cache.k_scales.cpu().numpy().copy()
        self.vs = cache.v_scales.cpu().numpy().copy()


def _at(P, D):
    t, d = np.meshgrid(np.arange(P), np.arange(D), indexing="ij")
    k = t // 16 * 16 * D + d // 64 * 1024 + t % 16 * 64 + d % 64
    v = t // 16 * 16 * D + d // 4 * 64 + t % 16 // 4 * 16 + d % 4 * 4 + t % 4
    return k, v


def _flat(pages):
    x = pages.cpu().float().double().numpy()
    return x.reshape(x.shape[0], x.shape[1], -1)


def unpack_k(pages):
    P, D = pages.shape[2] * 16, pages.shape[3] * 64
    return _flat(pages)[:, :, _at(P, D)[0]]


def unpack_v(pages):
    P, D = pages.shape[2] * 16, pages.shape[3] * 4
    return _flat(pages)[:, :, _at(P, D)[1]]


def to_e4m3(x):
    """float64 -> the nearest e4m3 value (ties to even), saturating."""
    _, e = np.frexp(x)
    step = np.exp2(np.maximum(e, -5) - 4.0)
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def new_scale(amax, fmt):
    """fp32 scale of a page whose largest finite magnitude is amax (fp32)."""
    if not amax > 0:
        return np.float32(0)
    if fmt == "int8":
        return max(np.float32(amax) / np.float32(127), MIN_SCALE)
    e = math.ceil(math.log2(float(amax) / 448.0))
    while float(amax) > 448.0 * 2.0 ** e:
        e += 1
    while float(amax) <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return max(np.float32(2.0 ** e), MIN_SCALE)


def encode(x, s, fmt):
    """fp32 values over the fp32 scale s, as code values."""
    if not s > 0:
        return np.zeros(x.shape)
    with np.errstate(invalid="ignore", over="ignore"):
        q = (x.astype(np.float32) / np.float32(s))
        if fmt == "int8":
            return np.nan_to_num(np.clip(np.rint(q), -127, 127), nan=0.0).astype(np.float64)
        return np.where(np.isnan(q), np.nan, to_e4m3(np.clip(q, -448, 448).astype(np.float64)))


def append(ref: Paged, x, which, table, lens, offs):
    """x: float64 [rows, H, D] (values of the call's dtype)."""
    codes, scales = (ref.k, ref.ks) if which == "k" else (ref.v, ref.vs)
    for s in range(len(lens)):
        n, L = offs[s + 1] - offs[s], lens[s]
        if L == 0:
            continue
        for slot in range((L - n) // ref.P, -(-L // ref.P)):
            lo, hi = max(L - n, slot * ref.P), min(L, (slot + 1) * ref.P)
            if lo >= hi:
                continue
            page = table[s][slot]
            for h in range(ref.H):
                new = x[offs[s] + lo - (L - n):offs[s] + hi - (L - n), h]
                fin = np.abs(new[np.isfinite(new)])
                s0 = scales[page, h] if lo > slot * ref.P else np.float32(0)
                s1 = max(s0, new_scale(np.float32(fin.max()) if fin.size else np.float32(0), ref.fmt))
                old = codes[page, h, :lo - slot * ref.P]
                if old.size and s1 > s0:
                    r = old.astype(np.float32) * (np.float32(s0) / np.float32(s1))
                    codes[page, h, :lo - slot * ref.P] = np.rint(r) if ref.fmt == "int8" else to_e4m3(r.astype(np.float64))
                codes[page, h, lo - slot * ref.P:hi - slot * ref.P] = encode(new, s1, ref.fmt)
                scales[page, h] = s1


def tokens(ref: Paged, which, table_row, lo, hi):
    """Dequantised values of tokens [lo, hi) of a sequence: float64 [hi - lo, H, D]."""
    codes, scales = (ref.k, ref.ks) if which == "k" else (ref.v, ref.vs)
    out = np.empty((hi - lo, ref.H, ref.D))
    for j in range(lo, hi):
        page = table_row[j // ref.P]
        out[j - lo] = codes[page, :, j % ref.P] * scales[page].astype(np.float64)[:, None]
    return out


def attention(ref: Paged, q, table, lens, offs, scale, causal=True, window=0):
    """q: float64 [rows, Hq, D] -> (out, lse, spread, score): the exact result,
    and per row and head what error bounds need: the largest over dimensions of
    sum p |v|, and the largest of scale * sum |q k|."""
    T, Hq, D = q.shape
    G = Hq // ref.H
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    spread, score = np.zeros((T, Hq)), np.zeros((T, Hq))
    for s in range(len(lens)):
        n, L = offs[s + 1] - offs[s], lens[s]
        if L == 0 or n == 0:
            continue
        k, v = tokens(ref, "k", table[s], 0, L), tokens(ref, "v", table[s], 0, L)
        pos = np.arange(L - n, L)[:, None]
        j = np.arange(L)[None, :]
        ok = np.ones((n, L), bool) if not causal else j <= pos
        if window:
            ok = ok & (j > pos - window)
        for h in range(Hq):
            qs = q[offs[s]:offs[s + 1], h]
            z = np.where(ok, qs @ k[:, h // G].T * scale, -np.inf)
            m = z.max(1, keepdims=True)
            p = np.exp(z - m)
            l = p.sum(1, keepdims=True)
            rows = slice(offs[s], offs[s + 1])
            out[rows, h] = p @ v[:, h // G] / l
            lse[rows, h] = (m + np.log(l))[:, 0]
            spread[rows, h] = (p @ np.abs(v[:, h // G]) / l).max(1)
            score[rows, h] = (np.where(ok, np.abs(qs) @ np.abs(k[:, h // G]).T * scale, 0.0)).max(1)
    return out, lse, spread, score


def rope(x, cos, sin, positions, axes, interleaved, inverse=False):
    """x float64 [rows, heads, D]; cos, sin [max_pos, half]; positions [n_axes, rows]."""
    half = cos.shape[1]
    y = x.copy()
    for i in range(half):
        p = positions[axes[i]]
        c, s = cos[p, i][:, None], sin[p, i][:, None] * (-1.0 if inverse else 1.0)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def make_batch(rng, news, befores, page, spare=3, room=2048):
    """(table int32 [S, max], lens, offs, num_pages): pages scattered, unused entries out of range; `room` columns
    more than needed (attention of several queries chooses its kernel by what a table has room for)."""
    lens = [a + b for a, b in zip(news, befores)]
    offs = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    per = [-(-x // page) for x in lens]
    num = sum(per) + spare
    order = rng.permutation(num)
    table = np.full((len(lens), max(per + [1]) + 1 + room), -7, np.int32)
    at = 0
    for s, c in enumerate(per):
        table[s, :c] = order[at:at + c]
        at += c
    return table, np.array(lens, np.int32), offs, num


def random_codes(rng, cache):
    """Fill a cache's pages with any finite codes and its scales with ordinary ones."""
    for t in (cache.k_pages, cache.v_pages):
        b = rng.integers(0, 256, t.numel(), dtype=np.uint8)
        if cache.fmt == "e4m3":
            b[(b & 0x7F) == 0x7F] = 0x3A  # no NaN
        else:
            b[b == 0x80] = 0x81  # -128 is not a code
        t.view(torch.uint8).view(-1).copy_(torch.from_numpy(b))
    for t in (cache.k_scales, cache.v_scales):
        e = rng.normal(size=t.shape).astype(np.float32)
        s = np.exp(0.3 * e) / 60 if cache.fmt == "int8" else np.exp2(np.rint(e) - 7)
        t.copy_(torch.from_numpy(s.astype(np.float32)))
