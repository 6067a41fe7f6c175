"""include/lora_attention.h on the host (no GPU needed): the entry points are
exported, their argument structures match the binding's, and what the host
refuses is refused before the device is touched."""

import ctypes
import os
import re

import pytest

from adapter_gemm_linear_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000  # an aligned address that a refused call never reads


@pytest.fixture(scope="module")
def L():
    from adapter_gemm_linear_gb300 import build
    build()
    return _lib.lib()


def test_exports_every_declared_symbol(L):
    text = open(os.path.join(ROOT, "include", "lora_attention.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = sorted(set(re.findall(r"\b(lora_[a-z0-9_]+)\s*\(", text)))
    assert sorted(n for n, _, _ in _lib.ATTENTION_SIGNATURES) == declared
    for name in declared:
        assert hasattr(L, name)


def test_pages_bytes(L):
    assert L.lora_kv_pages_bytes(3, 8, 128, 16) == 3 * 8 * 128 * 16
    assert L.lora_kv_pages_bytes(1 << 20, 64, 128, 128) == (1 << 20) * 64 * 128 * 128
    assert L.lora_kv_pages_bytes(0, 8, 128, 16) == 0


def rope_args(**kw):
    h = lambda p=P: _lib.Heads(p, 512, 128)  # noqa: E731
    a = dict(dtype=0, rows=4, head_dim=128, rot_dim=128, num_q_heads=4, num_k_heads=2, q=h(), q_out=h(), k=h(),
             k_out=h(), cos_table=P, sin_table=P, max_pos=16, num_axes=1, positions=P, pair_axis=None, interleaved=0,
             inverse=0)
    a.update(kw)
    return _lib.RopeArgs(**a)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), "LORA_ERR_DTYPE"), (dict(rows=-1), "LORA_ERR_INVALID_ARG"),
    (dict(head_dim=0), "LORA_ERR_INVALID_ARG"), (dict(head_dim=132), "LORA_ERR_ALIGNMENT"),
    (dict(rot_dim=136), "LORA_ERR_INVALID_ARG"), (dict(rot_dim=8), "LORA_ERR_INVALID_ARG"),
    (dict(rot_dim=72), "LORA_ERR_ALIGNMENT"), (dict(num_q_heads=0), "LORA_ERR_INVALID_ARG"),
    (dict(num_k_heads=-1), "LORA_ERR_INVALID_ARG"), (dict(num_axes=0), "LORA_ERR_INVALID_ARG"),
    (dict(num_axes=5), "LORA_ERR_INVALID_ARG"), (dict(max_pos=0), "LORA_ERR_INVALID_ARG"),
    (dict(cos_table=None), "LORA_ERR_INVALID_ARG"), (dict(positions=P + 2), "LORA_ERR_ALIGNMENT"),
    (dict(q=_lib.Heads(P + 8, 512, 128)), "LORA_ERR_ALIGNMENT"), (dict(q=_lib.Heads(P, 513, 128)), "LORA_ERR_ALIGNMENT"),
    (dict(k=_lib.Heads(None, 512, 128)), "LORA_ERR_INVALID_ARG"), (dict(q_out=_lib.Heads(P, -512, 128)), "LORA_ERR_INVALID_ARG"),
    (dict(pair_axis=bytes([0] * 63 + [1])), "LORA_ERR_INVALID_ARG"),
])
def test_rope_refusals(L, change, status):
    a = rope_args(**change)
    assert L.lora_rope(ctypes.byref(a), None) == _lib.STATUS[status]


def test_rope_without_rows_is_a_no_op(L):
    a = rope_args(rows=0, q=_lib.Heads(None, 512, 128), cos_table=None)
    assert L.lora_rope(ctypes.byref(a), None) == 0
    assert L.lora_rope(None, None) == _lib.STATUS["LORA_ERR_INVALID_ARG"]


def cache_desc(**kw):
    a = dict(format=0, num_pages=4, num_heads=2, head_dim=128, page_tokens=16, k_pages=P, v_pages=P, k_scales=P,
             v_scales=P)
    a.update(kw)
    return _lib.KvCacheDesc(**a)


def batch(**kw):
    a = dict(num_seqs=2, rows=3, seq_lens=P, offsets=P, block_table=P, max_pages=4)
    a.update(kw)
    return _lib.KvBatch(**a)


CACHE_CHANGES = [
    (dict(format=2), "LORA_ERR_UNSUPPORTED"), (dict(num_pages=0), "LORA_ERR_INVALID_ARG"),
    (dict(num_heads=0), "LORA_ERR_INVALID_ARG"), (dict(num_heads=5000), "LORA_ERR_UNSUPPORTED"),
    (dict(head_dim=96), "LORA_ERR_UNSUPPORTED"), (dict(page_tokens=8), "LORA_ERR_UNSUPPORTED"),
    (dict(page_tokens=256), "LORA_ERR_UNSUPPORTED"), (dict(k_pages=None), "LORA_ERR_INVALID_ARG"),
    (dict(v_scales=P + 4), "LORA_ERR_ALIGNMENT"),
]
BATCH_CHANGES = [
    (dict(num_seqs=-1), "LORA_ERR_INVALID_ARG"), (dict(rows=-1), "LORA_ERR_INVALID_ARG"),
    (dict(max_pages=0), "LORA_ERR_INVALID_ARG"), (dict(offsets=None), "LORA_ERR_INVALID_ARG"),
    (dict(seq_lens=None), "LORA_ERR_INVALID_ARG"), (dict(block_table=P + 2), "LORA_ERR_ALIGNMENT"),
]


@pytest.mark.parametrize("which,change,status", [("cache",) + c for c in CACHE_CHANGES] +
                         [("batch",) + c for c in BATCH_CHANGES])
def test_cache_and_batch_refusals(L, which, change, status):
    c = cache_desc(**(change if which == "cache" else {}))
    b = batch(**(change if which == "batch" else {}))
    h = _lib.Heads(P, 256, 128)
    want = _lib.STATUS[status]
    for fn in (L.lora_kv_append, L.lora_kv_gather):
        assert fn(ctypes.byref(c), ctypes.byref(b), 0, ctypes.byref(h), ctypes.byref(h), None) == want
    a = attention_args()
    assert L.lora_kv_attention(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a), None) == want
    assert L.lora_kv_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a)) == 0


@pytest.mark.parametrize("dtype,k,status", [
    (3, _lib.Heads(P, 256, 128), "LORA_ERR_DTYPE"), (0, _lib.Heads(None, 256, 128), "LORA_ERR_INVALID_ARG"),
    (0, _lib.Heads(P, 252, 128), "LORA_ERR_ALIGNMENT"), (1, _lib.Heads(P + 4, 256, 128), "LORA_ERR_ALIGNMENT"),
])
def test_rows_refusals(L, dtype, k, status):
    c, b, v = cache_desc(), batch(), _lib.Heads(P, 256, 128)
    for fn in (L.lora_kv_append, L.lora_kv_gather):
        assert fn(ctypes.byref(c), ctypes.byref(b), dtype, ctypes.byref(k), ctypes.byref(v), None) == _lib.STATUS[status]
        assert fn(ctypes.byref(c), ctypes.byref(b), 0, ctypes.byref(v), None, None) == _lib.STATUS["LORA_ERR_INVALID_ARG"]


def attention_args(**kw):
    a = dict(dtype=0, num_q_heads=8, q=_lib.Heads(P, 1024, 128), out=_lib.Heads(P, 1024, 128), lse=None, scale=0.1,
             causal=1, window=0, max_queries=2, workspace=P, workspace_bytes=0)
    a.update(kw)
    return _lib.AttentionArgs(**a)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=9), "LORA_ERR_DTYPE"), (dict(num_q_heads=0), "LORA_ERR_INVALID_ARG"),
    (dict(num_q_heads=7), "LORA_ERR_UNSUPPORTED"), (dict(num_q_heads=130), "LORA_ERR_UNSUPPORTED"),
    (dict(scale=0.0), "LORA_ERR_INVALID_ARG"), (dict(scale=float("nan")), "LORA_ERR_INVALID_ARG"),
    (dict(scale=float("inf")), "LORA_ERR_INVALID_ARG"), (dict(window=-1), "LORA_ERR_INVALID_ARG"),
    (dict(max_queries=0), "LORA_ERR_INVALID_ARG"), (dict(q=_lib.Heads(P, 1020, 128)), "LORA_ERR_ALIGNMENT"),
    (dict(out=_lib.Heads(None, 1024, 128)), "LORA_ERR_INVALID_ARG"), (dict(lse=P + 2), "LORA_ERR_ALIGNMENT"),
    (dict(workspace_bytes=0), "LORA_ERR_WORKSPACE"), (dict(workspace=None, workspace_bytes=1 << 40), "LORA_ERR_WORKSPACE"),
    (dict(workspace=P + 8, workspace_bytes=1 << 40), "LORA_ERR_ALIGNMENT"),
])
def test_attention_refusals(L, change, status):
    c, b, a = cache_desc(), batch(), attention_args(**change)
    assert L.lora_kv_attention(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a), None) == _lib.STATUS[status]


def test_calls_without_rows_or_sequences_are_no_ops(L):
    c, h = cache_desc(), _lib.Heads(None, 256, 128)
    for b in (batch(num_seqs=0, rows=0, seq_lens=None, block_table=None), batch(rows=0, seq_lens=None)):
        for fn in (L.lora_kv_append, L.lora_kv_gather):
            assert fn(ctypes.byref(c), ctypes.byref(b), 0, ctypes.byref(h), ctypes.byref(h), None) == 0
        a = attention_args(q=h, out=h, workspace_bytes=0)
        assert L.lora_kv_attention(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a), None) == 0
