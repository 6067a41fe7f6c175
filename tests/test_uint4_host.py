"""The 4-bit cache on the host (no GPU needed): sizes, the layout's restatement, and refusals."""

import ctypes

import numpy as np
import pytest
import torch

import uint4_reference as U
from adapter_gemm_linear_gb300 import KvCache, _lib, kv_pages_bytes, kv_scales_bytes
from test_attention_binding import Where
from test_attention_host import BATCH_CHANGES, L, attention_args, batch, cache_desc  # noqa: F401


def test_bytes(L):  # noqa: F811
    assert L.lora_kv_codes_bytes(4, 3, 8, 128, 16) == 3 * 8 * 128 * 16 // 2
    assert L.lora_kv_scales_bytes(4, 3, 8, 128, 16) == 3 * 8 * 16 * 2 * 4
    assert L.lora_kv_codes_bytes(0, 1 << 20, 64, 128, 128) == (1 << 20) * 64 * 128 * 128
    assert L.lora_kv_codes_bytes(4, 1 << 20, 64, 128, 128) == (1 << 19) * 64 * 128 * 128
    assert L.lora_kv_scales_bytes(1, 5, 7, 64, 16) == 5 * 7 * 4
    for fn in (L.lora_kv_codes_bytes, L.lora_kv_scales_bytes):
        assert fn(4, 0, 8, 128, 16) == 0 and fn(2, 1, 8, 128, 16) == 0
    assert kv_pages_bytes(3, 8, 64, 32) == 2 * kv_pages_bytes(3, 8, 64, 32, "uint4") == 3 * 8 * 64 * 32
    assert kv_scales_bytes(3, 8, 64, 32) == 96
    with pytest.raises(ValueError, match="uint4"):
        kv_pages_bytes(3, 8, 64, 32, "uint8")


@pytest.mark.parametrize("change,status", [
    (dict(format=3), "LORA_ERR_UNSUPPORTED"), (dict(format=5), "LORA_ERR_UNSUPPORTED"), (dict(head_dim=96), "LORA_ERR_UNSUPPORTED"),
    (dict(page_tokens=8), "LORA_ERR_UNSUPPORTED"), (dict(k_scales=None), "LORA_ERR_INVALID_ARG"),
    (dict(k_scales=0x10008), "LORA_ERR_ALIGNMENT"), (dict(v_pages=0x10001), "LORA_ERR_ALIGNMENT"),
])
def test_refusals(L, change, status):  # noqa: F811
    c = cache_desc(**{"format": 4, **change})
    b, h, a = batch(), _lib.Heads(0x10000, 256, 128), attention_args()
    for fn in (L.lora_kv_append, L.lora_kv_gather):
        assert fn(ctypes.byref(c), ctypes.byref(b), 0, ctypes.byref(h), ctypes.byref(h), None) == _lib.STATUS[status]
    assert L.lora_kv_attention(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a), None) == _lib.STATUS[status]


@pytest.mark.parametrize("change,status", BATCH_CHANGES)
def test_batch_refusals(L, change, status):  # noqa: F811
    c, b, h = cache_desc(format=4), batch(**change), _lib.Heads(0x10000, 256, 128)
    for fn in (L.lora_kv_append, L.lora_kv_gather):
        assert fn(ctypes.byref(c), ctypes.byref(b), 0, ctypes.byref(h), ctypes.byref(h), None) == _lib.STATUS[status]


def test_buffers_are_checked():
    shapes = dict(k_pages=(4, 2, 1, 1, 32, 16), v_pages=(4, 2, 1, 1, 32, 16), k_scales=(4, 2, 1, 1, 16, 2), v_scales=(4, 2, 1, 1, 16, 2))
    types = dict(k_pages=torch.uint8, v_pages=torch.uint8, k_scales=torch.float16, v_scales=torch.float16)
    good = {n: Where("cuda:0", s, types[n]) for n, s in shapes.items()}
    KvCache(4, 2, 64, 16, "uint4", **good)
    for name in shapes:
        for bad in (Where("cuda:0", shapes[name][:-1] + (4,), types[name]), Where("cuda:0", shapes[name], torch.int8),
                    Where("cuda:1", shapes[name], types[name])):
            with pytest.raises(ValueError):
                KvCache(4, 2, 64, 16, "uint4", device="cuda:0", **{**good, name: bad})


def test_the_restatement_of_the_layout():
    """Every place of a tile is used once, and a token's share of 16 bytes is whole bytes (nothing is read to write it)."""
    for D in (64, 128):
        for byte, _ in U.places(D).values():
            for t in range(16):
                mine = set(byte[t])
                assert all(mine.isdisjoint(byte[u]) for u in range(16) if u != t)
    c, s = U.quantise(np.arange(64, dtype=np.float32))
    assert s[0] == np.float16(4.2) and s[1] == 0 and c[0] == 0 and c[63] == 15
