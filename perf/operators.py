"""The measured cases of the operators between the q/k/v projections and the o
projection: rotary positions (rope), an 8-bit paged key/value cache written
(write) and read back (read), and attention over it (attention).

Rows of a batch belong to sequences: sequence s has rows offsets[s] up to
offsets[s + 1], the last of its seq_lens[s] tokens.  The cache keeps pages of
`page` tokens; a page of one head is stored in tiles of 16 tokens:

    k_pages [pages, heads, page/16, head_dim/64, 16 tokens, 64 dims]
    v_pages [pages, heads, page/16, head_dim/4, 4 token quads, 4 dims, 4 tokens]

with one fp32 scale per page and head in k_scales and v_scales.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
MIN_SCALE = 2.0 ** -120


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one decode step's q and k of 64 requests, a model of 32 query heads (hidden 4096): the smallest call
        dict(name="rope_decode", op="rope", rows=64, q_heads=32, kv_heads=8, head_dim=128, axes=1, interleaved=False,
             max_pos=8192, dtype="bf16"),
        # an image-and-text prompt of 8192 tokens with time, height and width positions, 64 query heads (hidden 8192)
        dict(name="rope_prompt_3axes", op="rope", rows=8192, q_heads=64, kv_heads=8, head_dim=128, axes=3,
             interleaved=False, max_pos=8192, dtype="bf16"),
        # one decode step of 256 requests writes a token each into pages that mostly hold older tokens
        dict(name="write_decode", op="write", seqs=256, rows=256, history=4096, history_max=8192, kv_heads=8,
             head_dim=128, page=16, fmt="int8", dtype="bf16", layout=1),
        # the prompts of 16 requests, 8192 tokens in ragged segments, written into fresh pages
        dict(name="write_prompts", op="write", seqs=16, rows=8192, history=0, history_max=0, kv_heads=8, head_dim=128,
             page=16, fmt="int8", dtype="bf16", layout=2),
        # one request's cache of some 1000 tokens read back (moved to another replica)
        dict(name="read_one", op="read", seqs=1, rows=1000, history=0, history_max=0, kv_heads=8, head_dim=128,
             page=16, fmt="e4m3", dtype="bf16", layout=3),
        # 64 requests' whole caches, 262144 tokens, read back
        dict(name="read_many", op="read", seqs=64, rows=262144, history=0, history_max=0, kv_heads=8, head_dim=128,
             page=64, fmt="int8", dtype="bf16", layout=4),
        # one interactive session: a single token against some 2000, latency is all
        dict(name="attn_decode_one", op="attention", seqs=1, rows=1, history=2000, history_max=2000, q_heads=32,
             kv_heads=8, head_dim=128, page=16, fmt="int8", dtype="bf16", causal=True, window=0, lse=False, layout=5),
        # the decode step of 256 requests of ragged lengths, 64 query heads on 8 key heads
        dict(name="attn_decode_256", op="attention", seqs=256, rows=256, history=4096, history_max=8192, q_heads=64,
             kv_heads=8, head_dim=128, page=16, fmt="int8", dtype="bf16", causal=True, window=0, lse=False, layout=6),
        # a decode step over four very long documents
        dict(name="attn_decode_long", op="attention", seqs=4, rows=4, history=131071, history_max=131071, q_heads=64,
             kv_heads=8, head_dim=128, page=64, fmt="e4m3", dtype="bf16", causal=True, window=0, lse=True, layout=7),
        # four drafted tokens a request checked at once, sliding window, heads of 64
        dict(name="attn_verify_window", op="attention", seqs=64, rows=256, history=4000, history_max=8000, q_heads=32,
             kv_heads=8, head_dim=64, page=32, fmt="e4m3", dtype="bf16", causal=True, window=1024, lse=False, layout=8),
        # prefill of 16 requests, 8192 tokens in ragged segments (the prompt that `write_prompts` wrote)
        dict(name="attn_prompts", op="attention", seqs=16, rows=8192, history=0, history_max=0, q_heads=64,
             kv_heads=8, head_dim=128, page=16, fmt="int8", dtype="bf16", causal=True, window=0, lse=False, layout=9),
        # a chunk of 2048 tokens of a long prompt whose first 32768 are cached: the largest
        dict(name="attn_chunk", op="attention", seqs=1, rows=2048, history=32768, history_max=32768, q_heads=32,
             kv_heads=8, head_dim=128, page=64, fmt="int8", dtype="bf16", causal=True, window=0, lse=True, layout=10),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attention", "attention", "attention"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    layout = rng.randrange(1000, 1 << 20)
    if op == "rope":
        kv = rng.choice([1, 2, 4, 8])
        return dict(op=op, rows=_log(rng, 1, 8192), q_heads=kv * rng.choice([1, 4, 8]), kv_heads=kv,
                    head_dim=rng.choice([64, 128]), axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.5,
                    max_pos=_log(rng, 64, 32768), dtype=dtype)
    c = dict(op=op, kv_heads=rng.choice([1, 2, 4, 8]), head_dim=rng.choice([64, 128]),
             page=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["int8", "e4m3"]), dtype=dtype, layout=layout)
    if op == "write":
        seqs = _log(rng, 1, 256)
        history = rng.choice([0, _log(rng, 1, 4096)])
        rows = rng.choice([seqs, max(seqs, _log(rng, seqs, 8192))])
        return dict(c, seqs=seqs, rows=rows, history=history, history_max=2 * history)
    if op == "read":
        seqs = _log(rng, 1, 64)
        return dict(c, seqs=seqs, rows=max(seqs, _log(rng, seqs, 131072)), history=0, history_max=0)
    c["q_heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 5, 8])
    c["window"] = rng.choice([0, 0, _log(rng, 16, 2048)])
    c["causal"] = True
    c["lse"] = rng.random() < 0.5
    kind = rng.choice(["decode", "decode", "verify", "prompts", "chunk"])
    small = dtype == "fp32"
    if kind == "decode":
        seqs = _log(rng, 1, 256)
        history = _log(rng, 1, max(2, min(16384, (65536 if small else 1048576) // seqs)))
        return dict(c, seqs=seqs, rows=seqs, history=history, history_max=2 * history)
    if kind == "verify":
        seqs = _log(rng, 1, 64)
        history = _log(rng, 1, 1024 if small else 8192)
        return dict(c, seqs=seqs, rows=seqs * rng.choice([2, 3, 4, 7]), history=history, history_max=2 * history)
    if kind == "prompts":
        seqs = _log(rng, 1, 16)
        causal = rng.random() < 0.8
        return dict(c, seqs=seqs, rows=max(seqs, _log(rng, 16, 512 if small else 8192 if causal else 4096)),
                    history=0, history_max=0, causal=causal)
    history = _log(rng, 64, 1024 if small else 12288)
    return dict(c, seqs=1, rows=_log(rng, 16, 128 if small else 2048), history=history, history_max=history)


def shape_of(case):
    """(rows, lengths) of each sequence; by the case alone, whatever the seed.
    With one row a sequence, or the same for all, they are even; else the rows
    are split in geometric segments."""
    r = random.Random(case["layout"])
    S, T = case["seqs"], case["rows"]
    if T % S == 0 and T // S <= 8:
        n = [T // S] * S
    else:
        w = [r.expovariate(1.0) + 0.02 for _ in range(S)]
        n = [max(1, int(T * x / sum(w))) for x in w]
        n[n.index(max(n))] += T - sum(n)
    if case["history"] == case["history_max"]:
        before = [case["history"]] * S
    else:
        before = [min(case["history_max"], int(r.expovariate(1.0 / max(1, case["history"])))) for _ in range(S)]
    return n, [a + b for a, b in zip(n, before)]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _codes(shape, fmt, gen):
    """Codes as quantised normal values have them: the block's largest is near the end of the range."""
    out = torch.empty(shape, dtype=CODES[fmt], device=DEV)
    flat = out.view(shape[0], -1)
    step = max(1, (1 << 27) // flat.shape[1])
    for i in range(0, shape[0], step):
        x = torch.randn(flat[i:i + step].shape, device=DEV, generator=gen)
        flat[i:i + step] = (x * 36.0).round_().clamp_(-127, 127).to(torch.int8) if fmt == "int8" else \
            (x * 100.0).clamp_(-448, 448).to(CODES[fmt])
    return out


def _scales(pages, heads, fmt, gen):
    z = torch.randn((pages, heads), device=DEV, generator=gen)
    return torch.exp(0.25 * z) / 36.0 if fmt == "int8" else torch.exp2((0.6 * z).round() - 7.0)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    H, D = case["kv_heads"], case["head_dim"]
    st = {"case": case}
    if case["op"] == "rope":
        T, n_axes, half = case["rows"], case["axes"], D // 2
        # q and k as the projections leave them: column ranges of one wider row
        qk = torch.randn((T, (case["q_heads"] + H) * D), device=DEV, generator=gen).to(dt)
        st["q"] = qk[:, :case["q_heads"] * D].view(T, case["q_heads"], D)
        st["k"] = qk[:, case["q_heads"] * D:].view(T, H, D)
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        angle = torch.arange(case["max_pos"], dtype=torch.float64, device=DEV)[:, None] * freq
        st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
        st["positions"] = torch.randint(0, case["max_pos"], (n_axes, T), device=DEV, generator=gen,
                                        dtype=torch.int32)
        # pairs in consecutive sections, one per axis, the first the shortest
        first = half // (n_axes + 1) if n_axes > 1 else half
        rest = half - first
        st["axes"] = [0] * first + [1 + i * (n_axes - 1) // rest for i in range(rest)]
        st["axis_index"] = torch.tensor(st["axes"], device=DEV)
        return st

    n, lens = shape_of(case)
    S, T, P = case["seqs"], case["rows"], case["page"]
    offs = [0]
    for x in n:
        offs.append(offs[-1] + x)
    per = [-(-x // P) for x in lens]
    pages = sum(per)
    # pages in random order, as a long-running server hands them out
    order = torch.randperm(pages, device=DEV, generator=gen, dtype=torch.int64).to(torch.int32)
    table = torch.full((S, max(per)), -1, dtype=torch.int32)
    flat, at = order.cpu(), 0
    for s in range(S):
        table[s, :per[s]] = flat[at:at + per[s]]
        at += per[s]
    st["block_table"], st["seq_lens"], st["offsets"] = table.to(DEV), _ints(lens), _ints(offs)
    st["k_pages"] = _codes((pages, H, P // 16, D // 64, 16, 64), case["fmt"], gen)
    st["v_pages"] = _codes((pages, H, P // 16, D // 4, 4, 4, 4), case["fmt"], gen)
    st["k_scales"], st["v_scales"] = _scales(pages, H, case["fmt"], gen), _scales(pages, H, case["fmt"], gen)
    if case["op"] == "write":
        kv = torch.randn((T, 2 * H * D), device=DEV, generator=gen).to(dt)
        st["k"], st["v"] = kv[:, :H * D].view(T, H, D), kv[:, H * D:].view(T, H, D)
        # what is read back: every page that the call writes to, from its start
        back = [x - (x - a) // P * P for x, a in zip(lens, n)]
        st["back_rows"] = sum(back)
        st["spread"] = max(-(-b // P) - (b - a) // P for a, b in zip(n, lens))  # pages that a sequence's rows touch
        offs = [0]
        for x in back:
            offs.append(offs[-1] + x)
        st["back_offsets"] = _ints(offs)
    elif case["op"] == "attention":
        q = torch.randn((T, case["q_heads"], D), device=DEV, generator=gen) * 2.0
        st["q"] = q.to(dt)
        st["max_queries"] = max(n)
    if own:  # the cache handle over these buffers, which a program makes once
        from adapter_gemm_linear_gb300 import KvCache
        st["cache"] = KvCache(pages, H, D, page_tokens=P, fmt=case["fmt"], k_pages=st["k_pages"],
                              v_pages=st["v_pages"], k_scales=st["k_scales"], v_scales=st["v_scales"])
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    case = st["case"]
    op = case["op"]
    if op == "rope":
        from adapter_gemm_linear_gb300 import rope
        q, k = rope(st["q"], st["k"], st["cos"], st["sin"], st["positions"], axes=st["axes"],
                    interleaved=case["interleaved"])
        return {"q": q, "k": k}
    cache = st["cache"]
    if op == "write":
        cache.append(st["k"], st["v"], st["block_table"], st["seq_lens"], st["offsets"])
        k, v = cache.gather(st["block_table"], st["seq_lens"], st["back_offsets"],
                            rows=st["back_rows"], dtype=DTYPES[case["dtype"]])
        return {"k": k, "v": v, "k_scales": st["k_scales"], "v_scales": st["v_scales"]}
    if op == "read":
        k, v = cache.gather(st["block_table"], st["seq_lens"], st["offsets"], rows=case["rows"],
                            dtype=DTYPES[case["dtype"]])
        return {"k": k, "v": v}
    r = cache.attention(st["q"], st["block_table"], st["seq_lens"], st["offsets"], max_queries=st["max_queries"],
                        causal=case["causal"], window=case["window"], return_lse=case["lse"])
    return {"out": r[0], "lse": r[1]} if case["lse"] else {"out": r}


def _rope_plain(x, cos, sin, interleaved):
    xf = x.float()
    half = x.shape[-1] // 2
    x1, x2 = (xf[..., 0::2], xf[..., 1::2]) if interleaved else (xf[..., :half], xf[..., half:])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack((y1, y2), -1).flatten(-2) if interleaved else torch.cat((y1, y2), -1)
    return y.to(x.dtype)


def _rows(offsets, lens, T):
    """Of each row: its sequence and its token's position."""
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(offsets, t, right=True) - 1
    return seq, (lens[seq] - offsets[seq + 1] + t).long()


def _k_tokens(pages):
    """[..., page/16, D/64, 16, 64] -> [..., page, D]"""
    return pages.transpose(-3, -2).flatten(-4, -3).flatten(-2)


def _k_tiles(x, like):
    return x.unflatten(-2, (-1, 16)).unflatten(-1, (-1, 64)).transpose(-3, -2).reshape(like)


def _v_tokens(pages):
    """[..., page/16, D/4, 4, 4, 4] -> [..., page, D]"""
    x = pages.movedim((-3, -1, -4, -2), (-4, -3, -2, -1))  # page/16, quad, token, D/4, dim
    return x.flatten(-5, -3).flatten(-2)


def _v_tiles(x, like):
    y = x.unflatten(-2, (-1, 4, 4)).unflatten(-1, (-1, 4))  # page/16, quad, token, D/4, dim
    return y.movedim((-4, -3, -2, -1), (-3, -1, -4, -2)).reshape(like)


def _scale_plain(amax, fmt):
    if fmt == "int8":
        s = (amax / torch.full_like(amax, 127.0)).clamp_min(MIN_SCALE)
    else:  # the least power of two s with amax <= 448 s
        m, e = torch.frexp(amax)
        s = torch.exp2((e - 9 + (m > 0.875).int()).to(amax.dtype)).clamp_min(MIN_SCALE)
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _append_plain(st, x, pages, scales, tokens, tiles, fmt):
    """Every page that new tokens touch, whole: its codes in hand, the new values over them, then quantised anew."""
    case = st["case"]
    P, lens, offs, table = case["page"], st["seq_lens"].long(), st["offsets"].long(), st["block_table"]
    n = offs[1:] - offs[:-1]
    first = (lens - n) // P
    last = (lens - 1) // P
    slot = torch.minimum(first[:, None] + torch.arange(st["spread"], device=DEV), last[:, None])  # [S, J]; the last repeated
    pid = table.gather(1, slot).long()
    pos = slot[:, :, None] * P + torch.arange(P, device=DEV)  # [S, J, P]
    start = (lens - n)[:, None, None]
    new = (pos >= start) & (pos < lens[:, None, None])
    row = (offs[:-1, None, None] + pos - start).clamp(0, x.shape[0] - 1)
    xf = x[row].float().movedim(3, 2)  # [S, J, H, P, D]
    newm = new[:, :, None, :, None]
    old_s = torch.where(slot[:, :, None] * P < start, scales[pid], torch.zeros((), device=DEV))  # [S, J, H]
    amax = torch.where(newm, xf.abs(), torch.zeros((), device=DEV)).amax((-1, -2))
    new_s = torch.maximum(old_s, _scale_plain(amax, fmt))
    div = torch.where(new_s > 0, new_s, torch.ones_like(new_s))[..., None, None]
    code = tokens(_pick(pages, pid)).float()
    ratio = old_s[..., None, None] / div
    if fmt == "int8":
        codes = torch.where(newm, torch.round(xf / div).clamp(-127, 127), torch.round(code * ratio))
    else:
        codes = torch.where(newm, xf / div, code * ratio)
    whole = tiles(codes.to(pages.dtype), pid.shape + pages.shape[1:])
    pages.view(torch.int8)[pid] = whole.view(torch.int8)
    scales[pid] = new_s


def _pick(pages, *at):
    return pages.view(torch.int8)[at].view(pages.dtype)


def _gather_plain(st, pages, scales, tokens, seq, pos, dtype):
    P = st["case"]["page"]
    pid = st["block_table"][seq, pos // P].long()
    # one token's codes, straight from its place in the tiles
    t = pos % P
    if tokens is _k_tokens:
        code = pages.view(torch.int8)[pid, :, t // 16, :, t % 16].flatten(-2)
    else:
        code = pages.view(torch.int8).movedim(-2, -1)[pid, :, t // 16, :, t % 16 // 4, t % 4].flatten(-2)
    code = code.contiguous().view(pages.dtype).float()
    return (code * scales[pid][:, :, None]).to(dtype)


def _attention_plain(st):
    case = st["case"]
    H, D, P, S = case["kv_heads"], case["head_dim"], case["page"], case["seqs"]
    G = case["q_heads"] // H
    lens, offs = st["seq_lens"].long(), st["offsets"].long()
    n = offs[1:] - offs[:-1]
    pid = st["block_table"].clamp_min(0).long()
    L = pid.shape[1] * P

    def values(pages, scales, tokens):  # [S, H, L, D]
        x = tokens(_pick(pages, pid)).float() * scales[pid][..., None, None]
        return x.transpose(1, 2).reshape(S, H, L, D)

    N = st["max_queries"]
    i = torch.arange(N, device=DEV)
    row = (offs[:-1, None] + i).clamp_max(st["q"].shape[0] - 1)
    q = st["q"][row].float().view(S, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, N * G, D)
    s = torch.matmul(q, values(st["k_pages"], st["k_scales"], _k_tokens).transpose(-1, -2))
    s *= 1.0 / math.sqrt(D)
    at = (lens - n)[:, None] + i  # [S, N]
    key = torch.arange(L, device=DEV)
    ok = key < lens[:, None, None]
    if case["causal"]:
        ok = ok & (key <= at[:, :, None])
    if case["window"]:
        ok = ok & (key > at[:, :, None] - case["window"])
    s.view(S, H, N, G, L).masked_fill_(~ok[:, None, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    s -= m
    s.exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, values(st["v_pages"], st["v_scales"], _v_tokens))
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = m + torch.log(total)

    seq, pos = _rows(st["offsets"], st["seq_lens"], st["q"].shape[0])
    idx = pos - (lens - n)[seq]

    def packed(x):  # [S, H, N * G, E] -> [T, H * G, E]
        return x.view(S, H, N, G, -1).permute(0, 2, 1, 3, 4)[seq, idx].flatten(1, 2)

    out = packed(o).to(st["q"].dtype)
    return {"out": out, "lse": packed(lse)[..., 0].contiguous()} if case["lse"] else {"out": out}


def _run_plain(st):
    case = st["case"]
    if case["op"] == "rope":
        p = st["positions"][st["axis_index"]].long().t()  # [T, half]
        cos, sin = st["cos"].gather(0, p)[:, None], st["sin"].gather(0, p)[:, None]
        return {"q": _rope_plain(st["q"], cos, sin, case["interleaved"]),
                "k": _rope_plain(st["k"], cos, sin, case["interleaved"])}
    if case["op"] == "attention":
        return _attention_plain(st)
    dt = DTYPES[case["dtype"]]
    offs, T = st["offsets"], case["rows"]
    if case["op"] == "write":
        _append_plain(st, st["k"], st["k_pages"], st["k_scales"], _k_tokens, _k_tiles, case["fmt"])
        _append_plain(st, st["v"], st["v_pages"], st["v_scales"], _v_tokens, _v_tiles, case["fmt"])
        offs, T = st["back_offsets"], st["back_rows"]
    seq, pos = _rows(offs, st["seq_lens"], T)
    out = {"k": _gather_plain(st, st["k_pages"], st["k_scales"], _k_tokens, seq, pos, dt),
           "v": _gather_plain(st, st["v_pages"], st["v_scales"], _v_tokens, seq, pos, dt)}
    if case["op"] == "write":
        out |= {"k_scales": st["k_scales"], "v_scales": st["v_scales"]}
    return out


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    eb = 4 if case["dtype"] == "fp32" else 2
    H, D = case["kv_heads"], case["head_dim"]
    if case["op"] == "rope":
        values = case["rows"] * (case["q_heads"] + H) * D
        table = min(case["max_pos"], case["rows"] * case["axes"]) * D // 2 * 8
        return {"bytes": values * 2 * eb + case["rows"] * case["axes"] * 4 + table, "flops": values * 3}
    n, lens = shape_of(case)
    P = case["page"]
    if case["op"] == "write":
        values = 2 * sum(n) * H * D
        back = [x - (x - a) // P * P for x, a in zip(lens, n)]
        old = 2 * (sum(back) - sum(n)) * H * D
        pages = sum(-(-b // P) for b in back)
        # rows read and codes written, older codes of their pages read; then all of these read and given back
        return {"bytes": values * (eb + 1) + old + (values + old) * (1 + eb) + 2 * pages * H * 8, "flops": 4 * values}
    if case["op"] == "read":
        values = 2 * sum(n) * H * D
        return {"bytes": values * (1 + eb) + 2 * sum(-(-x // P) for x in lens) * H * 4, "flops": values}
    pairs = keys = pages = 0
    w = case["window"]
    for a, b in zip(n, lens):
        lo = max(0, b - a + 1 - w) if w else 0  # the first key that any row sees
        keys += b - lo
        pages += -(-b // P) - lo // P
        for pos in range(b - a, b):
            top = pos + 1 if case["causal"] else b
            pairs += top - (max(0, pos + 1 - w) if w else 0)
    q = sum(n) * case["q_heads"] * D
    return {"bytes": 2 * keys * H * D + 2 * pages * H * 4 + pages * 4 + 2 * q * eb
            + (sum(n) * case["q_heads"] * 4 if case["lse"] else 0), "flops": 4 * pairs * case["q_heads"] * D}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _logical(st, name):
    """The whole cache of one tensor as [pages, page, H, D] in 64 bits, token by token from the stored layout."""
    c = st["case"]
    x = st[name + "_pages"].to(torch.float32).double()
    NP, H, P, D = x.shape[0], c["kv_heads"], c["page"], c["head_dim"]
    t, d = torch.arange(P, device=DEV)[:, None], torch.arange(D, device=DEV)[None, :]
    flat = x.reshape(NP, H, P * D)
    if name == "k":
        at = t // 16 * 16 * D + d // 64 * 1024 + t % 16 * 64 + d % 64
    else:
        at = t // 16 * 16 * D + d // 4 * 64 + t % 16 // 4 * 16 + d % 4 * 4 + t % 4
    return flat[:, :, at.flatten()].view(NP, H, P, D).transpose(1, 2)


def _exact_tokens(st, codes, scales, s, lo, hi):
    """Tokens lo..hi of sequence s: [hi - lo, H, D]."""
    P = st["case"]["page"]
    pos = torch.arange(lo, hi, device=DEV)
    pid = st["block_table"][s, pos // P].long()
    return codes[pid, pos % P] * scales[pid][:, :, None]


def _exact_write(st, name):
    """(values of the touched pages, scales) after the call."""
    c = st["case"]
    n, lens = shape_of(c)
    P, x = c["page"], st[name].double()
    codes, scales = _logical(st, name), st[name + "_scales"].double()
    row, out = 0, []
    for s, (a, b) in enumerate(zip(n, lens)):
        for slot in range((b - a) // P, -(-b // P)):
            lo, hi = max(b - a, slot * P), min(b, slot * P + P)
            pid = int(st["block_table"][s, slot])
            new = x[row + lo - (b - a):row + hi - (b - a)]  # [tokens, H, D]
            amax = new.abs().amax((0, 2))
            if c["fmt"] == "int8":
                fresh = (amax / 127.0).clamp_min(MIN_SCALE)
            else:
                fresh = torch.exp2(torch.ceil(torch.log2(amax / 448.0))).clamp_min(MIN_SCALE)
            fresh = torch.where(amax > 0, fresh, torch.zeros_like(fresh))
            old = scales[pid].clone() if lo > slot * P else torch.zeros_like(fresh)
            scale = torch.maximum(old, fresh)
            safe = torch.where(scale > 0, scale, torch.ones_like(scale))[None, :, None]
            value = torch.cat((codes[pid, :lo - slot * P] * old[None, :, None], new)) / safe
            if c["fmt"] == "int8":
                value = torch.round(value).clamp(-127, 127)
            else:  # three bits after the leading one, steps of 2^-9 below 2^-6
                e = torch.frexp(value)[1].clamp_min(-5).double()
                value = torch.round(value * torch.exp2(4 - e)) * torch.exp2(e - 4)
            out.append(value * scale[None, :, None])
            scales[pid] = scale
        row += a
    return torch.cat(out), scales


def exact(case, seed):
    if case["op"] == "attention" and work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    D = case["head_dim"]
    if case["op"] == "rope":
        half, out = D // 2, {}
        cos = torch.stack([st["cos"].double()[st["positions"][a].long(), i] for i, a in enumerate(st["axes"])], 1)
        sin = torch.stack([st["sin"].double()[st["positions"][a].long(), i] for i, a in enumerate(st["axes"])], 1)
        z = torch.complex(cos, sin)[:, None]
        for name in ("q", "k"):
            x = st[name].double()
            if case["interleaved"]:
                y = torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:2], half, 2).contiguous()) * z)
                out[name] = y.reshape(x.shape)
            else:
                y = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * z
                out[name] = torch.cat((y.real, y.imag), -1)
        return out
    n, lens = shape_of(case)
    if case["op"] == "write":
        if sum(-(-b // case["page"]) - (b - a) // case["page"] for a, b in zip(n, lens)) > 4096:
            return None
        k, ks = _exact_write(st, "k")
        v, vs = _exact_write(st, "v")
        return {"k": k, "v": v, "k_scales": ks, "v_scales": vs}
    if case["op"] == "read":
        out = {}
        for name in ("k", "v"):
            codes, scales = _logical(st, name), st[name + "_scales"].double()
            out[name] = torch.cat([_exact_tokens(st, codes, scales, s, b - a, b)
                                   for s, (a, b) in enumerate(zip(n, lens))])
        return out
    G = case["q_heads"] // case["kv_heads"]
    kc, ks = _logical(st, "k"), st["k_scales"].double()
    vc, vs = _logical(st, "v"), st["v_scales"].double()
    out, lses, row = [], [], 0
    for s, (a, b) in enumerate(zip(n, lens)):
        k, v = _exact_tokens(st, kc, ks, s, 0, b), _exact_tokens(st, vc, vs, s, 0, b)
        o = torch.empty((a, case["q_heads"], D), dtype=torch.float64, device=DEV)
        z = torch.empty((a, case["q_heads"]), dtype=torch.float64, device=DEV)
        pos = torch.arange(b - a, b, device=DEV)[:, None]
        j = torch.arange(b, device=DEV)[None, :]
        ok = j <= pos if case["causal"] else j >= 0
        if case["window"]:
            ok = ok & (j > pos - case["window"])
        for h in range(case["q_heads"]):
            x = st["q"][row:row + a, h].double() @ k[:, h // G].t() / math.sqrt(D)
            x = torch.where(ok, x, torch.full_like(x, -math.inf))
            z[:, h] = torch.logsumexp(x, 1)
            o[:, h] = torch.softmax(x, 1) @ v[:, h // G]
        out.append(o)
        lses.append(z)
        row += a
    return {"out": torch.cat(out), "lse": torch.cat(lses)} if case["lse"] else {"out": torch.cat(out)}
