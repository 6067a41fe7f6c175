"""PyTorch-facing binding of include/lora_attention.h: rotary positions, with
norms of queries and keys or without, the paged key/value cache of 8 or 4 bits,
and attention over it.

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

import ctypes
import math
import struct
from typing import Optional, Sequence, Tuple

import torch

from . import _lib
from ._lib import LORA_BLOCK_ROWS
from .api import LoraError, lora_dtype

_GROWTHS = {"least": _lib.KV_GROW_LEAST, "doubling": _lib.KV_GROW_DOUBLING}
_FORMATS = {"int8": (_lib.KV_INT8, torch.int8), "e4m3": (_lib.KV_E4M3, torch.float8_e4m3fn),
            "uint4": (_lib.KV_UINT4, torch.uint8)}

# A decode step makes these calls once per layer with a few microseconds of
# work each, so the argument structures of include/lora_attention.h are packed
# in one go (ctypes takes a microsecond for every few fields it sets) and the
# stream is asked for as a bare handle.
_ROPE_ARGS = struct.Struct("@6i PqqPqqPqqPqq PPiiPPii")
_NORM_ARGS = struct.Struct("@PPiifi")  # (what follows the lora_rope_args_t)
_NORM_GRADS = struct.Struct("@PqqPqqPPPN")
_BATCH = struct.Struct("@iiPPPi0P")
_HEADS = struct.Struct("@Pqq")
_ATTENTION_ARGS = struct.Struct("@iiPqqPqqPfiiiPN")
assert _ROPE_ARGS.size == ctypes.sizeof(_lib.RopeArgs) and _BATCH.size == ctypes.sizeof(_lib.KvBatch)
assert _ROPE_ARGS.size + _NORM_ARGS.size == ctypes.sizeof(_lib.NormRopeArgs)
assert _NORM_GRADS.size == ctypes.sizeof(_lib.NormRopeGrads)
assert _HEADS.size == ctypes.sizeof(_lib.Heads) and _ATTENTION_ARGS.size == ctypes.sizeof(_lib.AttentionArgs)

_DTYPES = {torch.bfloat16: _lib.LORA_BF16, torch.float32: _lib.LORA_FP32}
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _heads(t: torch.Tensor, name: str, device: int) -> Tuple[int, int, int]:
    strides = t.stride()
    if len(strides) != 3 or (strides[2] != 1 and t.numel() > 0):
        raise ValueError(f"{name} must be [rows, heads, head_dim] with contiguous heads")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected device {device}")
    return t.data_ptr(), strides[0], strides[1]


def _index(t: torch.Tensor, name: str, device: int) -> int:
    if t.dtype != torch.int32 or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name} must be contiguous int32 on device {device}")
    return t.data_ptr()


def _dtype(t: torch.dtype) -> int:
    code = _DTYPES.get(t)
    return lora_dtype(t) if code is None else code  # (lora_dtype says what is wrong)


def _call(status: int, what: str) -> None:
    if status != 0:
        raise LoraError(status, what)


def _elsewhere(f, device: int, stream: Optional[torch.cuda.Stream], args, **kw):
    """f(*args, **kw) with `device` current and, if given, on `stream`: outputs
    come from that stream's memory, and the caller's tensors are kept until it
    has passed the call."""
    if stream is None:
        with torch.cuda.device(device):
            return f(*args, **kw)
    if stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, the call's tensors on device {device}")
    with torch.cuda.stream(stream):
        result = f(*args, **kw)
    for t in list(args) + list(kw.values()):
        for x in (t.k_pages, t.v_pages, t.k_scales, t.v_scales) if isinstance(t, KvCache) else (t,):
            if isinstance(x, torch.Tensor):
                x.record_stream(stream)
    return result


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
    ``inverse`` turns the other way: the gradient of the call, or its undoing.
    ``stream``: launch there instead of on the current stream."""
    device = q.get_device()
    if device < 0:
        raise ValueError(f"q must be on a CUDA device, not on {q.device}")
    if stream is not None or device != _current_device():
        return _elsewhere(rope, device, stream, (q, k, cos, sin, positions), axes=axes, interleaved=interleaved,
                          inverse=inverse, q_out=q_out, k_out=k_out)
    args, q_out, k_out, _keep = _rope_args(q, k, cos, sin, positions, axes, interleaved, inverse, q_out, k_out, device)
    _call(_lib.lib().lora_rope(args, _current_stream(device)), "lora_rope")
    return q_out, k_out


def _rope_args(q, k, cos, sin, positions, axes, interleaved, inverse, q_out, k_out, device):
    """(lora_rope_args_t as bytes, q_out, k_out, what has to live until the call)"""
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q must be [rows, q_heads, head_dim]")
    rows, q_heads, D = shape
    table = cos.shape
    if len(table) != 2 or sin.shape != table or cos.dtype != torch.float32 or sin.dtype != torch.float32 or \
            not cos.is_contiguous() or not sin.is_contiguous() or cos.get_device() != device or sin.get_device() != device:
        raise ValueError(f"cos and sin must be contiguous float32 [max_pos, rot_dim/2] on device {device}")
    if positions.dim() not in (1, 2) or positions.shape[-1] != rows:
        raise ValueError("positions must be [rows] or [axes, rows]")
    if axes is not None and len(axes) != table[1]:
        raise ValueError(f"axes must name one axis for each of the {table[1]} pairs")
    if q_out is None:
        q_out = torch.empty(shape, dtype=q.dtype, device=q.device)
    elif q_out.shape != shape or q_out.dtype != q.dtype:
        raise ValueError("q_out must have q's shape and dtype")
    k_heads, kh, koh = 0, (0, 0, 0), (0, 0, 0)
    if k is not None:
        k_shape = k.shape
        if k.dtype != q.dtype or len(k_shape) != 3 or k_shape[0] != rows or k_shape[2] != D:
            raise ValueError("k must be [rows, k_heads, head_dim] with q's dtype, rows and head_dim")
        k_heads = k_shape[1]
        if k_out is None:
            k_out = torch.empty(k_shape, dtype=q.dtype, device=q.device)
        elif k_out.shape != k_shape or k_out.dtype != q.dtype:
            raise ValueError("k_out must have k's shape and dtype")
        kh, koh = _heads(k, "k", device), _heads(k_out, "k_out", device)
    pair_axis = None if axes is None else bytes(axes)
    axis_ptr = 0 if axes is None else ctypes.cast(pair_axis, ctypes.c_void_p).value
    return _ROPE_ARGS.pack(
        _dtype(q.dtype), rows, D, 2 * table[1], q_heads, k_heads, *_heads(q, "q", device),
        *_heads(q_out, "q_out", device), *kh, *koh, cos.data_ptr(), sin.data_ptr(), table[0],
        1 if positions.dim() == 1 else positions.shape[0], _index(positions, "positions", device), axis_ptr,
        interleaved, inverse), q_out, k_out if k is not None else None, pair_axis


def _norm_args(q, k, q_weight, k_weight, eps, unit_offset, device):
    """The rest of lora_norm_rope_args_t as bytes."""
    w = [t for t in (q_weight, k_weight if k is not None else None) if t is not None]
    for t in w:
        if t.shape != q.shape[2:] or t.dtype != w[0].dtype or not t.is_contiguous() or t.get_device() != device:
            raise ValueError(f"q_weight and k_weight must be contiguous [{q.shape[2]}] of one dtype on device {device}")
    return _NORM_ARGS.pack(0 if q_weight is None else q_weight.data_ptr(),
                           0 if k_weight is None or k is None else k_weight.data_ptr(),
                           _dtype(w[0].dtype) if w else _lib.LORA_FP32, unit_offset, eps, 0)


def norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], q_weight: Optional[torch.Tensor],
              k_weight: Optional[torch.Tensor], cos: torch.Tensor, sin: torch.Tensor, positions: torch.Tensor,
              eps: float = 1e-6, unit_offset: bool = False, axes: Optional[Sequence[int]] = None,
              interleaved: bool = False, q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """lora_norm_rope: every head of q and k (or None) divided by the root of
    its mean square + ``eps``, times its weight, and turned by its row's
    position, in one pass -> (q_out, k_out), new tensors unless given
    (``q_out=q`` works in place).

    ``q_weight``, ``k_weight``: [head_dim], bfloat16 or float32, or None for
    none; with ``unit_offset`` they are taken as 1 + weight.  The others: as
    rope.  head_dim up to 256."""
    device = q.get_device()
    if device < 0:
        raise ValueError(f"q must be on a CUDA device, not on {q.device}")
    if stream is not None or device != _current_device():
        return _elsewhere(norm_rope, device, stream, (q, k, q_weight, k_weight, cos, sin, positions), eps=eps,
                          unit_offset=unit_offset, axes=axes, interleaved=interleaved, q_out=q_out, k_out=k_out)
    args, q_out, k_out, _keep = _rope_args(q, k, cos, sin, positions, axes, interleaved, False, q_out, k_out, device)
    args += _norm_args(q, k, q_weight, k_weight, eps, unit_offset, device)
    _call(_lib.lib().lora_norm_rope(args, _current_stream(device)), "lora_norm_rope")
    return q_out, k_out


_norm_workspace = {}  # bytes of a backward call's workspace, by head_dim and device


def norm_rope_backward(dq: torch.Tensor, dk: Optional[torch.Tensor], q: torch.Tensor, k: Optional[torch.Tensor],
                       q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor], cos: torch.Tensor,
                       sin: torch.Tensor, positions: torch.Tensor, eps: float = 1e-6, unit_offset: bool = False,
                       axes: Optional[Sequence[int]] = None, interleaved: bool = False,
                       q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """lora_norm_rope_backward: from the gradients dq, dk of norm_rope's outputs
    -> (gradient of q, of k, of q_weight, of k_weight).  The other arguments are
    norm_rope's, but q_out and k_out, where the gradients of q and k go
    (``q_out=dq`` works in place).  Those of the weights are float32 [head_dim];
    None for what was None."""
    device = q.get_device()
    if device < 0:
        raise ValueError(f"q must be on a CUDA device, not on {q.device}")
    if stream is not None or device != _current_device():
        return _elsewhere(norm_rope_backward, device, stream, (dq, dk, q, k, q_weight, k_weight, cos, sin, positions),
                          eps=eps, unit_offset=unit_offset, axes=axes, interleaved=interleaved, q_out=q_out,
                          k_out=k_out, workspace=workspace)
    args, q_out, k_out, _keep = _rope_args(q, k, cos, sin, positions, axes, interleaved, False, q_out, k_out, device)
    args += _norm_args(q, k, q_weight, k_weight, eps, unit_offset, device)
    if dq.shape != q.shape or dq.dtype != q.dtype:
        raise ValueError("dq must have q's shape and dtype")
    if (dk is None) != (k is None) or (k is not None and (dk.shape != k.shape or dk.dtype != k.dtype)):
        raise ValueError("dk must have k's shape and dtype")
    L = _lib.lib()
    has_q, has_k = q_weight is not None, k_weight is not None and k is not None
    D = q.shape[2]
    dq_weight = torch.empty(D, dtype=torch.float32, device=q.device) if has_q else None
    dk_weight = torch.empty(D, dtype=torch.float32, device=q.device) if has_k else None
    if workspace is None:
        need = 0
        if has_q or has_k:
            need = _norm_workspace.get((D, device))  # (it depends on these alone)
            if need is None:
                need = L.lora_norm_rope_backward_workspace_bytes(args)
                if need:  # (0: arguments that the call will refuse)
                    _norm_workspace[D, device] = need
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {q.device}")
    grads = _NORM_GRADS.pack(*_heads(dq, "dq", device), *((0, 0, 0) if dk is None else _heads(dk, "dk", device)),
                             dq_weight.data_ptr() if has_q else 0, dk_weight.data_ptr() if has_k else 0, workspace.data_ptr(),
                             workspace.numel() * workspace.element_size())
    _call(L.lora_norm_rope_backward(args, grads, _current_stream(device)), "lora_norm_rope_backward")
    return q_out, k_out, dq_weight, dk_weight


def kv_pages_bytes(num_pages: int, num_heads: int, head_dim: int, page_tokens: int, fmt: str = "int8") -> int:
    """lora_kv_codes_bytes: device bytes of a cache's K codes (as many again for V)."""
    return int(_lib.lib().lora_kv_codes_bytes(_format(fmt)[0], num_pages, num_heads, head_dim, page_tokens))


def kv_scales_bytes(num_pages: int, num_heads: int, head_dim: int, page_tokens: int, fmt: str = "int8") -> int:
    """lora_kv_scales_bytes: device bytes of a cache's K scales (as many again for V)."""
    return int(_lib.lib().lora_kv_scales_bytes(_format(fmt)[0], num_pages, num_heads, head_dim, page_tokens))


def _format(fmt: str):
    if fmt not in _FORMATS:
        raise ValueError(f"unknown format {fmt!r}; use 'int8', 'e4m3' or 'uint4'")
    return _FORMATS[fmt]


class KvCache:
    """One layer's paged key/value cache (lora_kv_cache_t).

    ``fmt`` "int8", "e4m3" or "uint4"; head_dim 64 or 128; pages of 16, 32, 64 or
    128 tokens.  The codes (k_pages, v_pages) and the scales, one per page and
    head, or for "uint4" a scale and a least value (float16) per token and 64
    dimensions, are torch tensors, allocated here unless given.  Which pages a
    sequence owns is the caller's business (block tables); a page's older
    content does not matter once its first token is written anew.

    ``growth``: how an int8 page's scale grows when a later token does not
    fit.  "least" takes the least scale that holds it, the finest steps for
    prompts written at once, but each growth rounds the page's older codes again;
    "doubling" takes the least power of two of its first one, which keeps
    pages that are filled token by token within one step.  (e4m3 rescales exactly,
    and uint4 has a scale for each token.)
    """

    def __init__(self, num_pages: int, num_heads: int, head_dim: int, page_tokens: int = LORA_BLOCK_ROWS,
                 fmt: str = "int8", device=None, k_pages: Optional[torch.Tensor] = None,
                 v_pages: Optional[torch.Tensor] = None, k_scales: Optional[torch.Tensor] = None,
                 v_scales: Optional[torch.Tensor] = None, growth: str = "least"):
        if growth not in _GROWTHS:
            raise ValueError(f"unknown growth {growth!r}; use 'least' or 'doubling'")
        code, dtype = _format(fmt)
        self.fmt, self.growth = fmt, growth
        self.num_pages, self.num_heads = int(num_pages), int(num_heads)
        self.head_dim, self.page_tokens = int(head_dim), int(page_tokens)
        if device is None:
            device = k_pages.device if k_pages is not None else "cuda"
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"a KvCache is on a CUDA device, not on {device}")
        tiles = (self.num_pages, self.num_heads, self.page_tokens // LORA_BLOCK_ROWS)

        def tensor(t, shape, dt, name):
            if t is None:
                return torch.zeros(shape, dtype=dt, device=device)
            if t.shape != shape or t.dtype != dt or not t.is_contiguous() or t.device.type != "cuda" or \
                    (device.index is not None and t.device != device):
                raise ValueError(f"{name} must be contiguous {dt} {tuple(shape)} on {device}")
            return t

        D = self.head_dim
        k_tile, v_tile, scales, scale_dtype = (D // 64, LORA_BLOCK_ROWS, 64), (D // 4, 4, 4, 4), tiles[:2], torch.float32
        if fmt == "uint4":
            k_tile = v_tile = (D // 64, 32, 16)
            scales, scale_dtype = tiles + (D // 64, LORA_BLOCK_ROWS, 2), torch.float16
        self.k_pages = tensor(k_pages, tiles + k_tile, dtype, "k_pages")
        device = self.k_pages.device  # ("cuda" names none: the other buffers are of k_pages' own)
        self.v_pages = tensor(v_pages, tiles + v_tile, dtype, "v_pages")
        self.k_scales = tensor(k_scales, scales, scale_dtype, "k_scales")
        self.v_scales = tensor(v_scales, scales, scale_dtype, "v_scales")
        self.device = self.k_pages.device
        self._device = self.k_pages.get_device()
        self._workspace = {}  # bytes of an attention call's workspace, by what they depend on
        self._desc = _lib.KvCacheDesc(code, self.num_pages, self.num_heads, D, self.page_tokens, _GROWTHS[growth],
                                      self.k_pages.data_ptr(), self.v_pages.data_ptr(), self.k_scales.data_ptr(),
                                      self.v_scales.data_ptr())
        self._ref = ctypes.byref(self._desc)

    def _batch(self, rows: int, block_table: torch.Tensor, seq_lens: torch.Tensor,
               offsets: Optional[torch.Tensor]) -> bytes:
        device, S = self._device, seq_lens.shape[0]
        table = block_table.shape
        if len(table) != 2 or table[0] != S:
            raise ValueError(f"block_table must be [{S}, max_pages]")
        if offsets is not None and offsets.shape != (S + 1,):
            raise ValueError(f"offsets must be [{S + 1}]")
        return _BATCH.pack(S, rows, _index(seq_lens, "seq_lens", device),
                           0 if offsets is None else _index(offsets, "offsets", device),
                           _index(block_table, "block_table", device), table[1])

    def _check(self, t: torch.Tensor, name: str) -> None:
        shape = t.shape
        if len(shape) != 3 or shape[1] != self.num_heads or shape[2] != self.head_dim:
            raise ValueError(f"{name} must be [rows, {self.num_heads}, {self.head_dim}]")

    def append(self, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
               offsets: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
        """lora_kv_append: quantise the rows' k and v [rows, num_heads, head_dim]
        into their sequences' pages, as the last tokens of seq_lens tokens.
        ``stream``: launch there instead of on the current stream."""
        device = self._device
        if stream is not None or device != _current_device():
            return _elsewhere(KvCache.append, device, stream, (self, k, v, block_table, seq_lens, offsets))
        self._check(k, "k")
        self._check(v, "v")
        if k.dtype != v.dtype or k.shape[0] != v.shape[0]:
            raise ValueError("k and v must have the same dtype and rows")
        _call(_lib.lib().lora_kv_append(
            self._ref, self._batch(k.shape[0], block_table, seq_lens, offsets), _dtype(k.dtype),
            _HEADS.pack(*_heads(k, "k", device)), _HEADS.pack(*_heads(v, "v", device)), _current_stream(device)),
            "lora_kv_append")

    def gather(self, block_table: torch.Tensor, seq_lens: torch.Tensor, offsets: Optional[torch.Tensor] = None,
               rows: Optional[int] = None, dtype: torch.dtype = torch.bfloat16, k_out: Optional[torch.Tensor] = None,
               v_out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """lora_kv_gather: the rows' keys and values, dequantised -> (k, v)
        [rows, num_heads, head_dim], new tensors of ``dtype`` unless given.
        ``rows`` (needed with offsets and no k_out) is offsets' last value.
        Rows of padding (length 0), of skipped sequences and of none are not
        written: in new tensors they hold whatever the memory held.
        ``stream``: launch there instead of on the current stream."""
        device = self._device
        if stream is not None or device != _current_device():
            return _elsewhere(KvCache.gather, device, stream, (self, block_table, seq_lens, offsets), rows=rows,
                              dtype=dtype, k_out=k_out, v_out=v_out)
        if k_out is not None:
            self._check(k_out, "k_out")
            rows, dtype = k_out.shape[0], k_out.dtype
        elif rows is None:
            if offsets is not None:
                raise ValueError("give rows (offsets' last value), or k_out and v_out")
            rows = seq_lens.shape[0]
        shape = (rows, self.num_heads, self.head_dim)
        if k_out is None:
            k_out = torch.empty(shape, dtype=dtype, device=self.device)
        if v_out is None:
            v_out = torch.empty(shape, dtype=dtype, device=self.device)
        elif v_out.shape != shape or v_out.dtype != dtype:
            raise ValueError("v_out must have k_out's shape and dtype")
        _call(_lib.lib().lora_kv_gather(
            self._ref, self._batch(rows, block_table, seq_lens, offsets), _dtype(dtype),
            _HEADS.pack(*_heads(k_out, "k_out", device)), _HEADS.pack(*_heads(v_out, "v_out", device)),
            _current_stream(device)), "lora_kv_gather")
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
        offsets, else all rows).  It and the block table's width, as a bound on
        the lengths, choose the kernel for bf16 queries: a table much wider than
        its longest sequence needs costs short calls of several queries some
        time, and the same call with another width may differ in its last bits.
        Of a "uint4" cache prompts take K's values rounded to 11 bits unless an
        lse is asked for: ask for it where keys lie far from 0 in all dimensions.
        ``window`` > 0 limits a query to the last ``window`` positions up to its
        own; ``scale`` defaults to head_dim^-0.5.
        ``stream``: launch there instead of on the current stream."""
        shape, device = q.shape, self._device
        if stream is not None or device != _current_device():
            return _elsewhere(KvCache.attention, device, stream, (self, q, block_table, seq_lens, offsets),
                              max_queries=max_queries, causal=causal, window=window, scale=scale,
                              return_lse=return_lse, out=out, lse=lse, workspace=workspace)
        if len(shape) != 3 or shape[2] != self.head_dim:
            raise ValueError(f"q must be [rows, q_heads, {self.head_dim}]")
        rows, Hq, _ = shape
        if max_queries is None:
            max_queries = 1 if offsets is None else max(1, rows)
        if scale is None:
            scale = 1.0 / math.sqrt(self.head_dim)
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=self.device)
        elif out.shape != shape or out.dtype != q.dtype:
            raise ValueError("out must have q's shape and dtype")
        if lse is None:
            if return_lse:
                lse = torch.empty((rows, Hq), dtype=torch.float32, device=self.device)
        elif lse.shape != (rows, Hq) or lse.dtype != torch.float32 or not lse.is_contiguous() \
                or lse.get_device() != device:
            raise ValueError(f"lse must be contiguous float32 [{rows}, {Hq}] on {self.device}")
        batch = self._batch(rows, block_table, seq_lens, offsets)
        head = (_dtype(q.dtype), Hq, *_heads(q, "q", device), *_heads(out, "out", device),
                0 if lse is None else lse.data_ptr(), scale, causal, window, max_queries)
        L = _lib.lib()
        if workspace is None:
            key = (head[0], Hq, max_queries, rows, block_table.shape, device)
            need = self._workspace.get(key)
            if need is None:
                need = L.lora_kv_attention_workspace_bytes(self._ref, batch, _ATTENTION_ARGS.pack(*head, 0, 0))
                if need:
                    if len(self._workspace) >= 256:  # (ever new numbers of rows)
                        self._workspace.clear()
                    self._workspace[key] = need
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=self.device)
        elif workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on {self.device}")
        _call(L.lora_kv_attention(self._ref, batch, _ATTENTION_ARGS.pack(
            *head, workspace.data_ptr(), workspace.numel() * workspace.element_size()), _current_stream(device)),
            "lora_kv_attention")
        return (out, lse) if lse is not None else out
