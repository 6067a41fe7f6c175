"""The measured cases of two groups of operators between the q/k/v projections
and the o projection: norms of queries and keys for each head with the rotary
positions in the same pass (norm_rope) and its gradient (norm_rope_grad), and
a paged key/value cache held in 4 bits: written (write), read back (read),
and attention over it (attention).

Rows of a batch belong to sequences: sequence s has rows offsets[s] up to
offsets[s + 1], the last of its seq_lens[s] tokens.  The cache keeps pages of
`page` tokens; a value is scale * code + least, codes 0 to 15, with a scale
and a least value in f16 for each 64 dimensions of a token and head.  A page
of one head is stored in tiles of 16 tokens, each 64 dimensions of a tile in
32 pieces of 16 bytes:

    k_pages [pages, heads, page/16, head_dim/64, 32 pieces, 16 bytes]
    v_pages like k_pages
    k_scales, v_scales [pages, heads, page/16, head_dim/64, 16 tokens, (scale, least)]

K: piece 4 g + q has dimensions 16 q .. 16 q + 15 of tokens t = 4 (g / 2) + g % 2
(its first 8 bytes) and t + 2.  Four bytes hold eight dimensions: 0 and 2, 4 and 6,
1 and 3, 5 and 7, low half of a byte first.
V: piece 4 g + q has tokens 4 q .. 4 q + 3; its four groups of four bytes are dimensions
4 g, 4 g + 2, 4 g + 32 and 4 g + 34 (low halves) and the next (high halves), the bytes
tokens 0, 2, 1, 3 of the four.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
LARGEST = 32768.0  # what the 4-bit cache holds at most


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one decode step's q and k of 64 requests, a model of 32 query heads (hidden 4096): the smallest call
        dict(name="norm_rope_decode", op="norm_rope", rows=64, q_heads=32, kv_heads=8, head_dim=128, axes=1,
             interleaved=False, unit_offset=False, max_pos=8192, dtype="bf16"),
        # an image-and-text prompt of 8192 tokens with time, height and width positions, 64 query heads (hidden 8192)
        dict(name="norm_rope_prompt_3axes", op="norm_rope", rows=8192, q_heads=64, kv_heads=8, head_dim=128, axes=3,
             interleaved=False, unit_offset=False, max_pos=8192, dtype="bf16"),
        # gradients of a short ragged batch, heads of 64
        dict(name="norm_rope_grad_short", op="norm_rope_grad", rows=333, q_heads=32, kv_heads=8, head_dim=64, axes=1,
             interleaved=True, unit_offset=True, max_pos=4096, dtype="bf16"),
        # gradients of 8192 tokens, 64 query heads
        dict(name="norm_rope_grad_8192", op="norm_rope_grad", rows=8192, q_heads=64, kv_heads=8, head_dim=128, axes=1,
             interleaved=False, unit_offset=False, max_pos=8192, dtype="bf16"),
        # one decode step of 256 requests writes a token each into pages that mostly hold older tokens
        dict(name="write4_decode", op="write", seqs=256, rows=256, history=4096, history_max=8192, kv_heads=8,
             head_dim=128, page=16, dtype="bf16", layout=1),
        # the prompts of 16 requests, 8192 tokens in ragged segments, written into fresh pages
        dict(name="write4_prompts", op="write", seqs=16, rows=8192, history=0, history_max=0, kv_heads=8, head_dim=128,
             page=16, dtype="bf16", layout=2),
        # one request's cache of some 1000 tokens read back (moved to another replica)
        dict(name="read4_one", op="read", seqs=1, rows=1000, history=0, history_max=0, kv_heads=8, head_dim=128,
             page=16, dtype="bf16", layout=3),
        # 64 requests' whole caches, 262144 tokens, read back
        dict(name="read4_many", op="read", seqs=64, rows=262144, history=0, history_max=0, kv_heads=8, head_dim=128,
             page=64, dtype="bf16", layout=4),
        # one interactive session: a single token against some 2000, latency is all
        dict(name="attn4_decode_one", op="attention", seqs=1, rows=1, history=2000, history_max=2000, q_heads=32,
             kv_heads=8, head_dim=128, page=16, dtype="bf16", causal=True, window=0, lse=False, layout=5),
        # the decode step of 256 requests of ragged lengths, 64 query heads on 8 key heads
        dict(name="attn4_decode_256", op="attention", seqs=256, rows=256, history=4096, history_max=8192, q_heads=64,
             kv_heads=8, head_dim=128, page=16, dtype="bf16", causal=True, window=0, lse=False, layout=6),
        # four drafted tokens a request checked at once, sliding window, heads of 64
        dict(name="attn4_verify_window", op="attention", seqs=64, rows=256, history=4000, history_max=8000, q_heads=32,
             kv_heads=8, head_dim=64, page=32, dtype="bf16", causal=True, window=1024, lse=True, layout=8),
        # a chunk of 2048 tokens of a long prompt whose first 32768 are cached: the largest
        dict(name="attn4_chunk", op="attention", seqs=1, rows=2048, history=32768, history_max=32768, q_heads=32,
             kv_heads=8, head_dim=128, page=64, dtype="bf16", causal=True, window=0, lse=True, layout=10),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "write", "read", "attention", "attention", "attention"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    layout = rng.randrange(1000, 1 << 20)
    if op.startswith("norm_rope"):
        kv = rng.choice([1, 2, 4, 8])
        return dict(op=op, rows=_log(rng, 1, 8192 if dtype == "bf16" else 4096), q_heads=kv * rng.choice([1, 4, 8]),
                    kv_heads=kv, head_dim=rng.choice([64, 128, 128, 256]) if kv < 8 else rng.choice([64, 128]),
                    axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.5, unit_offset=rng.random() < 0.3,
                    max_pos=_log(rng, 64, 32768), dtype=dtype)
    c = dict(op=op, kv_heads=rng.choice([1, 2, 4, 8]), head_dim=rng.choice([64, 128]),
             page=rng.choice([16, 32, 64, 128]), dtype=dtype, layout=layout)
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


def _codes(shape, gen):
    """Codes as quantised normal values have them: 64 of them spread over the whole range."""
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    flat = out.view(shape[0], -1)
    step = max(1, (1 << 26) // flat.shape[1])
    for i in range(0, shape[0], step):
        x = torch.randn((2,) + flat[i:i + step].shape, device=DEV, generator=gen)
        x = (x * 3.1 + 7.5).round_().clamp_(0, 15)
        flat[i:i + step] = (x[0] + 16.0 * x[1]).to(torch.uint8)
    return out


def _scales(shape, gen):
    """(scale, least) as 64 normal values have them, tokens of varying magnitude."""
    x = torch.empty(shape, dtype=torch.float16, device=DEV)
    size = torch.exp(0.25 * torch.randn(shape[:-1], device=DEV, generator=gen))
    x[..., 0] = size * 0.32
    x[..., 1] = size * (-2.4 + 0.3 * torch.randn(shape[:-1], device=DEV, generator=gen))
    return x


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    H, D = case["kv_heads"], case["head_dim"]
    st = {"case": case}

    def rows_of_heads(rows, std=1.0):
        # q and k as the projections leave them: column ranges of one wider row
        qk = (torch.randn((rows, (case["q_heads"] + H) * D), device=DEV, generator=gen) * std).to(dt)
        return qk[:, :case["q_heads"] * D].view(rows, case["q_heads"], D), qk[:, case["q_heads"] * D:].view(rows, H, D)

    if case["op"].startswith("norm_rope"):
        T, n_axes, half = case["rows"], case["axes"], D // 2
        st["q"], st["k"] = rows_of_heads(T, 3.0)
        if case["op"] == "norm_rope_grad":
            st["dq"], st["dk"] = rows_of_heads(T)
        for name in ("q_weight", "k_weight"):
            w = 0.2 * torch.randn((D,), device=DEV, generator=gen) + (0.0 if case["unit_offset"] else 1.0)
            st[name] = w.to(dt)
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
    for name in ("k", "v"):
        st[name + "_pages"] = _codes((pages, H, P // 16, D // 64, 32, 16), gen)
        st[name + "_scales"] = _scales((pages, H, P // 16, D // 64, 16, 2), gen)
    if case["op"] == "write":
        kv = torch.randn((T, 2 * H * D), device=DEV, generator=gen).to(dt)
        st["k"], st["v"] = kv[:, :H * D].view(T, H, D), kv[:, H * D:].view(T, H, D)
        # what is read back: every page that the call writes to, from its start
        back = [x - (x - a) // P * P for x, a in zip(lens, n)]
        st["back_rows"] = sum(back)
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
        st["cache"] = KvCache(pages, H, D, page_tokens=P, fmt="uint4", k_pages=st["k_pages"],
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
    if op.startswith("norm_rope"):
        from adapter_gemm_linear_gb300 import norm_rope, norm_rope_backward
        args = (st["q"], st["k"], st["q_weight"], st["k_weight"], st["cos"], st["sin"], st["positions"])
        kw = dict(eps=EPS, unit_offset=case["unit_offset"], axes=st["axes"], interleaved=case["interleaved"])
        if op == "norm_rope":
            q, k = norm_rope(*args, **kw)
            return {"q": q, "k": k}
        dq, dk, dqw, dkw = norm_rope_backward(st["dq"], st["dk"], *args, **kw)
        return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
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


def _rotate(x, cos, sin, interleaved):
    half = x.shape[-1] // 2
    x1, x2 = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    return torch.stack((y1, y2), -1).flatten(-2) if interleaved else torch.cat((y1, y2), -1)


def _norm_rope_plain(st, name, cos, sin):
    case, x = st["case"], st[name]
    xf = x.float()
    w = st[name + "_weight"].float() + (1.0 if case["unit_offset"] else 0.0)
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
    if case["op"] == "norm_rope":
        return _rotate(xf * r * w, cos, sin, case["interleaved"]).to(x.dtype)
    h = _rotate(st["d" + name].float(), cos, -sin, case["interleaved"])
    a = h * w
    dx = r * (a - xf * (r * r * (a * xf).mean(-1, keepdim=True)))
    return dx.to(x.dtype), (h * xf * r).sum((0, 1))


def _rows(offsets, lens, T):
    """Of each row: its sequence and its token's position."""
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(offsets, t, right=True) - 1
    return seq, (lens[seq] - offsets[seq + 1] + t).long()


def _halves(pages):
    """[..., 32, 16] bytes -> [..., 32, 16, (low, high)]"""
    return torch.stack((pages & 15, pages >> 4), -1)


def _tokens(pages, scales, name):
    """Codes and scales of whole pages [..., page/16, D/64, ...] -> values [..., page, D]"""
    x = _halves(pages)
    lead = x.dim() - 5  # before page/16
    if name == "k":  # pieces (quad, parity, 16 dims), bytes (pair, half of 16, 2, 2)
        x = x.unflatten(-3, (4, 2, 4)).unflatten(-2, (2, 2, 2, 2))
        tokens, dims = (2, 5, 3), (1, 4, 6, 8, 9, 7)  # tile, 64 dims, quad, parity, dims 16, pair, half, b1, b0, high
    else:  # pieces (4 dims, quad), bytes (half of 64, 2 dims, 2, 2)
        x = x.unflatten(-3, (8, 4)).unflatten(-2, (2, 2, 2, 2))
        tokens, dims = (3, 7, 6), (1, 4, 2, 5, 8)
    x = x.permute(*range(lead), lead, *(lead + i for i in tokens + dims))
    x = x.flatten(lead + 4).flatten(lead + 1, lead + 3)  # [..., page/16, 16, D]
    s = scales.float().movedim(-2, -3)  # [..., page/16, 16, D/64, 2]
    v = x.unflatten(-1, (-1, 64)).float() * s[..., :1] + s[..., 1:]
    return v.flatten(-2).flatten(-3, -2)


def _place(name, t, d):
    """Byte of (token, dimension) within a tile, and whether it is the high half."""
    if name == "k":
        e = d % 8
        piece = (t // 4 * 2 + t % 2) * 4 + d % 64 // 16
        return d // 64 * 512 + piece * 16 + t // 2 % 2 * 8 + d % 16 // 8 * 4 + e % 2 * 2 + e // 4, e // 2 % 2
    piece = d % 32 // 4 * 4 + t // 4
    return d // 64 * 512 + piece * 16 + (d % 64 // 32 * 2 + d % 4 // 2) * 4 + t % 2 * 2 + t % 4 // 2, d % 2


def _gather_plain(st, name, seq, pos, dtype):
    P, H, D = st["case"]["page"], st["case"]["kv_heads"], st["case"]["head_dim"]
    pages, scales = st[name + "_pages"], st[name + "_scales"]
    out = torch.empty((seq.shape[0], H, D), dtype=dtype, device=DEV)
    d = torch.arange(D, device=DEV)
    for i in range(0, seq.shape[0], 16384):
        p = pos[i:i + 16384]
        pid = st["block_table"][seq[i:i + 16384], p // P].long()
        t = p % P
        tile = pages.view(*pages.shape[:3], -1)[pid, :, t // 16]  # [rows, H, bytes]
        byte, high = _place(name, t[:, None] % 16, d)
        code = tile.gather(2, byte[:, None, :].expand(-1, H, -1)).int()
        code = torch.where(high.bool()[:, None] if high.dim() == 2 else high.bool(), code >> 4, code & 15).float()
        s = scales[pid, :, t // 16, :, t % 16].float()  # [rows, H, D/64, 2]
        out[i:i + 16384] = (code.unflatten(-1, (-1, 64)) * s[..., :1] + s[..., 1:]).flatten(-2).to(dtype)
    return out


def _append_plain(st, name):
    case = st["case"]
    P, H, D = case["page"], case["kv_heads"], case["head_dim"]
    pages, scales = st[name + "_pages"], st[name + "_scales"]
    seq, pos = _rows(st["offsets"], st["seq_lens"], case["rows"])
    pid = st["block_table"][seq, pos // P].long()
    x = st[name].float().unflatten(-1, (-1, 64))  # [rows, H, D/64, 64]
    x = torch.where(x == x, x, torch.zeros((), device=DEV))
    finite = x.abs() < math.inf
    x = torch.where(finite, x.clamp(-LARGEST, LARGEST), x)
    lo = torch.where(finite, x, math.inf).amin(-1)
    hi = torch.where(finite, x, -math.inf).amax(-1)
    lo, hi = (torch.where(finite.any(-1), y, torch.zeros((), device=DEV)) for y in (lo, hi))
    least, scale = lo.half(), ((hi - lo) / 15.0).half()
    s = scale.float()[..., None]
    code = torch.where(s > 0, torch.round(((x - least.float()[..., None]) / s).clamp(0, 15)), 0.0).to(torch.uint8)
    code = code.flatten(-2)
    t = pos % P
    scales[pid, :, t // 16, :, t % 16] = torch.stack((scale, least), -1)
    # the two halves of a byte are dimensions of the same token
    flat = pages.view(*pages.shape[:3], -1)
    d = torch.arange(D, device=DEV)
    _, high = _place(name, torch.zeros((), dtype=torch.int64, device=DEV), d)
    low_d, high_d = d[high == 0], d[high == 1]
    byte_low = _place(name, t[:, None] % 16, low_d)[0]
    byte_high = _place(name, t[:, None] % 16, high_d)[0]
    order = byte_high[0].argsort()[byte_low[0].argsort().argsort()]  # the high half beside each low one
    both = code[:, :, low_d] | (code[:, :, high_d[order]] << 4)
    rows = torch.arange(H, device=DEV)[None, :, None]
    flat[pid[:, None, None], rows, (t // 16)[:, None, None], byte_low[:, None, :]] = both


def _attention_plain(st):
    case = st["case"]
    H, D, P, S = case["kv_heads"], case["head_dim"], case["page"], case["seqs"]
    G = case["q_heads"] // H
    lens, offs = st["seq_lens"].long(), st["offsets"].long()
    n = offs[1:] - offs[:-1]
    pid = st["block_table"].clamp_min(0).long()
    L = pid.shape[1] * P

    def values(name):  # [S, H, L, D]
        x = _tokens(st[name + "_pages"][pid], st[name + "_scales"][pid], name)
        return x.transpose(1, 2).reshape(S, H, L, D)

    N = st["max_queries"]
    i = torch.arange(N, device=DEV)
    row = (offs[:-1, None] + i).clamp_max(st["q"].shape[0] - 1)
    q = st["q"][row].float().view(S, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, N * G, D)
    s = torch.matmul(q, values("k").transpose(-1, -2))
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
    o = torch.matmul(s, values("v"))
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
    if case["op"].startswith("norm_rope"):
        p = st["positions"][st["axis_index"]].long().t()  # [T, half]
        cos, sin = st["cos"].gather(0, p)[:, None], st["sin"].gather(0, p)[:, None]
        q, k = _norm_rope_plain(st, "q", cos, sin), _norm_rope_plain(st, "k", cos, sin)
        if case["op"] == "norm_rope":
            return {"q": q, "k": k}
        return {"dq": q[0], "dk": k[0], "dq_weight": q[1], "dk_weight": k[1]}
    if case["op"] == "attention":
        return _attention_plain(st)
    dt = DTYPES[case["dtype"]]
    offs, T = st["offsets"], case["rows"]
    if case["op"] == "write":
        _append_plain(st, "k")
        _append_plain(st, "v")
        offs, T = st["back_offsets"], st["back_rows"]
    seq, pos = _rows(offs, st["seq_lens"], T)
    out = {"k": _gather_plain(st, "k", seq, pos, dt), "v": _gather_plain(st, "v", seq, pos, dt)}
    if case["op"] == "write":
        out |= {"k_scales": st["k_scales"], "v_scales": st["v_scales"]}
    return out


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    eb = 4 if case["dtype"] == "fp32" else 2
    H, D = case["kv_heads"], case["head_dim"]
    if case["op"].startswith("norm_rope"):
        grad = case["op"] == "norm_rope_grad"
        values = case["rows"] * (case["q_heads"] + H) * D
        table = min(case["max_pos"], case["rows"] * case["axes"]) * D // 2 * 8
        return {"bytes": values * (3 if grad else 2) * eb + case["rows"] * case["axes"] * 4 + table
                + 2 * D * (eb + (4 if grad else 0)), "flops": values * (14 if grad else 7)}
    n, lens = shape_of(case)
    P = case["page"]
    stored = 0.5 + 4 / 64  # bytes a value
    if case["op"] == "write":
        values = 2 * sum(n) * H * D
        back = 2 * sum(x - (x - a) // P * P for x, a in zip(lens, n)) * H * D
        # rows read and codes written; then the touched pages read and given back
        return {"bytes": values * (eb + stored) + back * (stored + eb), "flops": 6 * values}
    if case["op"] == "read":
        values = 2 * sum(n) * H * D
        return {"bytes": values * (stored + eb), "flops": 2 * values}
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
    return {"bytes": 2 * keys * H * D * stored + pages * 4 + 2 * q * eb
            + (sum(n) * case["q_heads"] * 4 if case["lse"] else 0), "flops": 4 * pairs * case["q_heads"] * D}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _logical(st, name):
    """Codes, scales and least values of the whole cache of one tensor, [pages, page, H, D] in 64 bits, byte by byte
    from the stored layout."""
    c = st["case"]
    x, s = st[name + "_pages"], st[name + "_scales"]
    NP, H, P, D = x.shape[0], c["kv_heads"], c["page"], c["head_dim"]
    where, high = [], []
    for t in range(16):
        for d in range(D):
            block, r = divmod(d, 64)
            if name == "k":
                g, second = 2 * (t // 4) + t % 2, t % 4 // 2
                word, e = divmod(r % 16, 8)
                nibble = (0, 4, 1, 5, 2, 6, 3, 7)[e]
                at = 512 * block + 16 * (4 * g + r // 16) + 8 * second + 4 * word
            else:
                word = 2 * (r // 32) + r % 4 // 2
                nibble = 2 * (0, 2, 1, 3)[t % 4] + r % 2
                at = 512 * block + 16 * (4 * (r % 32 // 4) + t // 4) + 4 * word
            where.append(at + nibble // 2)
            high.append(nibble % 2)
    flat = x.reshape(NP, H, P // 16, 8 * D)[..., torch.tensor(where, device=DEV)].to(torch.int16)
    codes = (flat >> (4 * torch.tensor(high, device=DEV, dtype=torch.int16))) % 16
    codes = codes.reshape(NP, H, P, D).transpose(1, 2).double()
    s = s.double().permute(0, 2, 4, 1, 3, 5).reshape(NP, P, H, D // 64, 2).repeat_interleave(64, 3)
    return codes, s[..., 0], s[..., 1]


def _exact_tokens(st, values, s, lo, hi):
    """Tokens lo..hi of sequence s: [hi - lo, H, D]."""
    P = st["case"]["page"]
    pos = torch.arange(lo, hi, device=DEV)
    return values[st["block_table"][s, pos // P].long(), pos % P]


def _to_f16(x):
    """64-bit values rounded to 11 significant bits, steps of 2^-24 at least."""
    e = torch.frexp(x)[1].clamp_min(-13).double()
    return torch.round(x * torch.exp2(11 - e)) * torch.exp2(e - 11)


def _exact_write(st, name):
    """(values of the touched pages, scales) after the call."""
    c = st["case"]
    n, lens = shape_of(c)
    P, x = c["page"], st[name].double()
    codes, scale, least = _logical(st, name)
    old = codes * scale + least
    scales = st[name + "_scales"].double()
    row, out = 0, []
    for s, (a, b) in enumerate(zip(n, lens)):
        first = (b - a) // P * P
        g = x[row:row + a].unflatten(-1, (-1, 64)).clamp(-LARGEST, LARGEST)  # [tokens, H, D/64, 64]
        m = _to_f16(g.amin(-1))
        step = _to_f16((g.amax(-1) - g.amin(-1)) / 15.0)
        safe = torch.where(step > 0, step, torch.ones_like(step))[..., None]
        q = torch.round((g - m[..., None]) / safe).clamp(0, 15)
        new = (q * step[..., None] + m[..., None]).flatten(-2)
        out.append(torch.cat((_exact_tokens(st, old, s, first, b - a), new)))
        pos = torch.arange(b - a, b, device=DEV)
        pid = st["block_table"][s, pos // P].long()
        scales[pid, :, pos % P // 16, :, pos % 16] = torch.stack((step, m), -1)
        row += a
    return torch.cat(out), scales


def exact(case, seed):
    if case["op"] == "attention" and work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    D = case["head_dim"]
    if case["op"].startswith("norm_rope"):
        half, out = D // 2, {}
        cos = torch.stack([st["cos"].double()[st["positions"][a].long(), i] for i, a in enumerate(st["axes"])], 1)
        sin = torch.stack([st["sin"].double()[st["positions"][a].long(), i] for i, a in enumerate(st["axes"])], 1)
        z = torch.complex(cos, sin)[:, None]

        def turn(x, z):
            if case["interleaved"]:
                y = torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:2], half, 2).contiguous()) * z)
                return y.reshape(x.shape)
            y = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * z
            return torch.cat((y.real, y.imag), -1)

        for name in ("q", "k"):
            x = st[name].double()
            w = st[name + "_weight"].double() + float(case["unit_offset"])
            rms = torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS)
            unit = x / rms
            if case["op"] == "norm_rope":
                out[name] = turn(unit * w, z)
                continue
            g = turn(st["d" + name].double(), z.conj())
            out["d" + name + "_weight"] = torch.einsum("thd,thd->d", g, unit)
            g = g * w
            out["d" + name] = (g - unit * (g * unit).sum(-1, keepdim=True) / D) / rms
        return out
    n, lens = shape_of(case)
    if case["op"] == "write":
        k, ks = _exact_write(st, "k")
        v, vs = _exact_write(st, "v")
        return {"k": k, "v": v, "k_scales": ks, "v_scales": vs}
    values = {}
    for name in ("k", "v"):
        codes, scale, least = _logical(st, name)
        values[name] = codes.mul_(scale).add_(least)
        del codes, scale, least
    if case["op"] == "read":
        return {name: torch.cat([_exact_tokens(st, values[name], s, b - a, b) for s, (a, b) in enumerate(zip(n, lens))])
                for name in ("k", "v")}
    G = case["q_heads"] // case["kv_heads"]
    out, lses, row = [], [], 0
    for s, (a, b) in enumerate(zip(n, lens)):
        k, v = _exact_tokens(st, values["k"], s, 0, b), _exact_tokens(st, values["v"], s, 0, b)
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
