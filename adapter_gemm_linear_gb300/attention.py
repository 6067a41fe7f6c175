"""PyTorch-facing binding of include/lora_attention.h: rotary positions, the
8-bit paged key/value cache and attention over it.

As in api.py, the functions only marshal arguments: torch allocates device
memory and provides the stream, the C library does the work, and an argument
that it refuses raises LoraError.  Names follow the header without the
``lora_`` prefix.

Rows and sequences: ``offsets`` (device int32 [num_seqs + 1]; None: one row
each) says which rows of a call belong to which sequence.  They are the last
tokens of a sequence of ``seq_lens[s]`` (device int32) tokens, the call's own
included, and ``block_table`` (device int32 [num_seqs, max_pages]) names the
pages that hold its tokens.
"""

from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional, Sequence, Tuple

import torch

from . import _lib
from ._lib import LORA_BLOCK_ROWS
from .api import LoraError, lora_dtype

_FORMATS = {"int8": (_lib.KV_INT8, torch.int8), "e4m3": (_lib.KV_E4M3, torch.float8_e4m3fn)}


def _heads(t: torch.Tensor, name: str, device: torch.device) -> _lib.Heads:
    if t.dim() != 3 or (t.stride(2) != 1 and t.numel() > 0):
        raise ValueError(f"{name} must be [rows, heads, head_dim] with contiguous heads")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return _lib.Heads(t.data_ptr(), t.stride(0), t.stride(1))


def _index(t: torch.Tensor, name: str, device: torch.device) -> int:
    if t.dtype != torch.int32 or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be contiguous int32 on {device}")
    return t.data_ptr()


@contextlib.contextmanager
def _launching(device: torch.device, stream: Optional[torch.cuda.Stream], tensors):
    """The handle of the stream to launch on, with it and the device current
    (so that outputs come from that stream's memory), and the caller's tensors
    kept until the stream has passed the call."""
    if stream is None:
        if device.index is None or device.index == torch.cuda.current_device():
            yield torch.cuda.current_stream().cuda_stream
        else:
            with torch.cuda.device(device):
                yield torch.cuda.current_stream().cuda_stream
        return
    with torch.cuda.stream(stream):
        yield stream.cuda_stream
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _call(status: int, what: str) -> None:
    if status != 0:
        raise LoraError(status, what)


def rope_tables(max_pos: int, rot_dim: int, base: float = 10000.0, device="cuda") -> Tuple[torch.Tensor, torch.Tensor]:
    """(cos, sin), float32 [max_pos, rot_dim/2] each: the angles p * base^(-2i/rot_dim),
    taken in 64 bits, so that long positions keep their phase."""
    i = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * base ** (-2.0 * i / rot_dim)
    return angle.cos().float(), angle.sin().float()


def rope(q: torch.Tensor, k: Optional[torch.Tensor], cos: torch.Tensor, sin: torch.Tensor, positions: torch.Tensor,
         axes: Optional[Sequence[int]] = None, interleaved: bool = False, inverse: bool = False,
         q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
         stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """lora_rope: q [rows, q_heads, D] and k [rows, k_heads, D] (or None)
    turned by their rows' positions -> (q_out, k_out), new tensors unless
    given (``q_out=q`` works in place).

    ``cos``/``sin``: float32 [max_pos, rot_dim/2] (rope_tables); ``positions``:
    int32 [rows], or [axes, rows] for positions of several axes (time, height,
    width), with ``axes[i]`` the axis of pair i (default: axis 0).
    ``inverse`` turns the other way: the gradient of the call, or its undoing."""
    device = q.device
    if cos.dtype != torch.float32 or cos.dim() != 2 or not cos.is_contiguous() or \
            sin.dtype != torch.float32 or sin.shape != cos.shape or not sin.is_contiguous():
        raise ValueError("cos and sin must be contiguous float32 [max_pos, rot_dim/2]")
    if cos.device != device or sin.device != device:
        raise ValueError(f"cos and sin must be on {device}")
    rows, D = int(q.shape[0]), int(q.shape[-1])
    if positions.dim() not in (1, 2) or positions.shape[-1] != rows:
        raise ValueError("positions must be [rows] or [axes, rows]")
    if axes is not None and len(axes) != cos.shape[1]:
        raise ValueError(f"axes must name one axis for each of the {cos.shape[1]} pairs")
    if k is not None and (k.dtype != q.dtype or k.shape[0] != rows or k.shape[-1] != D):
        raise ValueError("k must have q's dtype, rows and head_dim")
    with _launching(device, stream, (q, k, cos, sin, positions, q_out, k_out)) as st:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=device)
        if k is not None and k_out is None:
            k_out = torch.empty(k.shape, dtype=q.dtype, device=device)
        for x, y, name in ((q, q_out, "q_out"), (k, k_out, "k_out")):
            if x is not None and (y.shape != x.shape or y.dtype != q.dtype):
                raise ValueError(f"{name} must have its input's shape and dtype")
        none = _lib.Heads(None, 0, 0)
        args = _lib.RopeArgs(
            lora_dtype(q.dtype), rows, D, 2 * int(cos.shape[1]), int(q.shape[1]), 0 if k is None else int(k.shape[1]),
            _heads(q, "q", device), _heads(q_out, "q_out", device),
            none if k is None else _heads(k, "k", device), none if k is None else _heads(k_out, "k_out", device),
            cos.data_ptr(), sin.data_ptr(), int(cos.shape[0]), 1 if positions.dim() == 1 else int(positions.shape[0]),
            _index(positions, "positions", device), None if axes is None else bytes(axes), int(interleaved),
            int(inverse))
        _call(_lib.lib().lora_rope(ctypes.byref(args), st), "lora_rope")
    return q_out, k_out if k is not None else None


def kv_pages_bytes(num_pages: int, num_heads: int, head_dim: int, page_tokens: int) -> int:
    """lora_kv_pages_bytes: device bytes of a cache's K codes (as many again for V)."""
    return int(_lib.lib().lora_kv_pages_bytes(num_pages, num_heads, head_dim, page_tokens))


class KvCache:
    """One layer's 8-bit paged key/value cache (lora_kv_cache_t).

    ``fmt`` "int8" or "e4m3"; head_dim 64 or 128; pages of 16, 32, 64 or 128
    tokens.  The codes (k_pages, v_pages) and the scales, one per page and
    head, are torch tensors, allocated here unless given.  Which pages a
    sequence owns is the caller's business (block tables); a page's older
    content does not matter once its first token is written anew.
    """

    def __init__(self, num_pages: int, num_heads: int, head_dim: int, page_tokens: int = LORA_BLOCK_ROWS,
                 fmt: str = "int8", device=None, k_pages: Optional[torch.Tensor] = None,
                 v_pages: Optional[torch.Tensor] = None, k_scales: Optional[torch.Tensor] = None,
                 v_scales: Optional[torch.Tensor] = None):
        if fmt not in _FORMATS:
            raise ValueError(f"unknown format {fmt!r}; use 'int8' or 'e4m3'")
        code, dtype = _FORMATS[fmt]
        self.fmt = fmt
        self.num_pages, self.num_heads = int(num_pages), int(num_heads)
        self.head_dim, self.page_tokens = int(head_dim), int(page_tokens)
        if device is None:
            device = k_pages.device if k_pages is not None else "cuda"
        device = torch.device(device)
        tiles = (self.num_pages, self.num_heads, self.page_tokens // LORA_BLOCK_ROWS)

        def tensor(t, shape, dt, name):
            if t is None:
                return torch.zeros(shape, dtype=dt, device=device)
            if t.shape != shape or t.dtype != dt or not t.is_contiguous() or t.device.type != device.type:
                raise ValueError(f"{name} must be contiguous {dt} {tuple(shape)} on {device}")
            return t

        D = self.head_dim
        self.k_pages = tensor(k_pages, tiles + (D // 64, LORA_BLOCK_ROWS, 64), dtype, "k_pages")
        self.v_pages = tensor(v_pages, tiles + (D // 4, 4, 4, 4), dtype, "v_pages")
        self.k_scales = tensor(k_scales, tiles[:2], torch.float32, "k_scales")
        self.v_scales = tensor(v_scales, tiles[:2], torch.float32, "v_scales")
        self.device = self.k_pages.device
        self._desc = _lib.KvCacheDesc(code, self.num_pages, self.num_heads, D, self.page_tokens,
                                      self.k_pages.data_ptr(), self.v_pages.data_ptr(), self.k_scales.data_ptr(),
                                      self.v_scales.data_ptr())
        self._ref = ctypes.byref(self._desc)

    def _batch(self, rows: int, block_table: torch.Tensor, seq_lens: torch.Tensor,
               offsets: Optional[torch.Tensor]) -> _lib.KvBatch:
        S = int(seq_lens.shape[0])
        if block_table.dim() != 2 or block_table.shape[0] != S:
            raise ValueError(f"block_table must be [{S}, max_pages]")
        if offsets is not None and offsets.shape != (S + 1,):
            raise ValueError(f"offsets must be [{S + 1}]")
        return _lib.KvBatch(S, rows, _index(seq_lens, "seq_lens", self.device),
                            None if offsets is None else _index(offsets, "offsets", self.device),
                            _index(block_table, "block_table", self.device), int(block_table.shape[1]))

    def _check(self, t: torch.Tensor, name: str) -> None:
        if t.dim() != 3 or t.shape[1:] != (self.num_heads, self.head_dim):
            raise ValueError(f"{name} must be [rows, {self.num_heads}, {self.head_dim}]")

    def append(self, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
               offsets: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
        """lora_kv_append: quantise the rows' k and v [rows, num_heads, head_dim]
        into their sequences' pages, as the last tokens of seq_lens tokens."""
        self._check(k, "k")
        self._check(v, "v")
        if k.dtype != v.dtype or k.shape[0] != v.shape[0]:
            raise ValueError("k and v must have the same dtype and rows")
        with _launching(self.device, stream, (k, v, block_table, seq_lens, offsets, self.k_pages, self.v_pages,
                                              self.k_scales, self.v_scales)) as st:
            b = self._batch(int(k.shape[0]), block_table, seq_lens, offsets)
            kh, vh = _heads(k, "k", self.device), _heads(v, "v", self.device)
            _call(_lib.lib().lora_kv_append(self._ref, ctypes.byref(b), lora_dtype(k.dtype), ctypes.byref(kh),
                                            ctypes.byref(vh), st), "lora_kv_append")

    def gather(self, block_table: torch.Tensor, seq_lens: torch.Tensor, offsets: Optional[torch.Tensor] = None,
               rows: Optional[int] = None, dtype: torch.dtype = torch.bfloat16, k_out: Optional[torch.Tensor] = None,
               v_out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """lora_kv_gather: the rows' keys and values, dequantised -> (k, v)
        [rows, num_heads, head_dim], new tensors of ``dtype`` unless given.
        ``rows`` (needed with offsets and no k_out) is offsets' last value."""
        if k_out is not None:
            self._check(k_out, "k_out")
            rows, dtype = int(k_out.shape[0]), k_out.dtype
        elif rows is None:
            if offsets is not None:
                raise ValueError("give rows (offsets' last value), or k_out and v_out")
            rows = int(seq_lens.shape[0])
        with _launching(self.device, stream, (block_table, seq_lens, offsets, k_out, v_out, self.k_pages,
                                              self.v_pages, self.k_scales, self.v_scales)) as st:
            shape = (rows, self.num_heads, self.head_dim)
            if k_out is None:
                k_out = torch.empty(shape, dtype=dtype, device=self.device)
            if v_out is None:
                v_out = torch.empty(shape, dtype=dtype, device=self.device)
            if v_out.shape != shape or v_out.dtype != dtype:
                raise ValueError("v_out must have k_out's shape and dtype")
            b = self._batch(rows, block_table, seq_lens, offsets)
            kh, vh = _heads(k_out, "k_out", self.device), _heads(v_out, "v_out", self.device)
            _call(_lib.lib().lora_kv_gather(self._ref, ctypes.byref(b), lora_dtype(dtype), ctypes.byref(kh),
                                            ctypes.byref(vh), st), "lora_kv_gather")
        return k_out, v_out

    def attention(self, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                  offsets: Optional[torch.Tensor] = None, max_queries: Optional[int] = None, causal: bool = True,
                  window: int = 0, scale: Optional[float] = None, return_lse: bool = False,
                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
        """lora_kv_attention: softmax attention of q [rows, q_heads, head_dim]
        over the sequences' cached keys and values -> out like q (and, with
        ``return_lse`` or ``lse`` given, the float32 [rows, q_heads] log of the
        softmax's sum).  The rows' own tokens must be in the cache.

        ``max_queries`` bounds the rows of one sequence (default: 1 without
        offsets, else all rows); ``window`` > 0 limits a query to the last
        ``window`` positions up to its own; ``scale`` defaults to head_dim^-0.5."""
        if q.dim() != 3 or q.shape[2] != self.head_dim:
            raise ValueError(f"q must be [rows, q_heads, {self.head_dim}]")
        rows, Hq = int(q.shape[0]), int(q.shape[1])
        if max_queries is None:
            max_queries = 1 if offsets is None else max(1, rows)
        if scale is None:
            scale = 1.0 / math.sqrt(self.head_dim)
        with _launching(self.device, stream, (q, block_table, seq_lens, offsets, out, lse, workspace, self.k_pages,
                                              self.v_pages, self.k_scales, self.v_scales)) as st:
            if out is None:
                out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
            elif out.shape != q.shape or out.dtype != q.dtype:
                raise ValueError("out must have q's shape and dtype")
            if lse is None:
                if return_lse:
                    lse = torch.empty((rows, Hq), dtype=torch.float32, device=self.device)
            elif lse.shape != (rows, Hq) or lse.dtype != torch.float32 or not lse.is_contiguous() \
                    or lse.device != self.device:
                raise ValueError(f"lse must be contiguous float32 [{rows}, {Hq}] on {self.device}")
            b = self._batch(rows, block_table, seq_lens, offsets)
            args = _lib.AttentionArgs(lora_dtype(q.dtype), Hq, _heads(q, "q", self.device),
                                      _heads(out, "out", self.device), None if lse is None else lse.data_ptr(),
                                      scale, int(causal), int(window), int(max_queries), None, 0)
            bref, aref = ctypes.byref(b), ctypes.byref(args)
            L = _lib.lib()
            if workspace is None:
                need = int(L.lora_kv_attention_workspace_bytes(self._ref, bref, aref))
                workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=self.device)
            args.workspace = workspace.data_ptr()
            args.workspace_bytes = workspace.numel() * workspace.element_size()
            _call(L.lora_kv_attention(self._ref, bref, aref, st), "lora_kv_attention")
        return (out, lse) if lse is not None else out
