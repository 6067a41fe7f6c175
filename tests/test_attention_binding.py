"""What attention.py refuses before anything reaches the device (no GPU needed)."""

import pytest
import torch

from adapter_gemm_linear_gb300 import KvCache, attention, rope


def test_rope_refuses_tensors_of_the_host():
    x = torch.zeros((2, 1, 64))
    table, pos = torch.zeros((4, 32)), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        rope(x, None, table, table, pos)
    with pytest.raises(ValueError, match="CUDA"):
        rope(x, x, table, table, pos, q_out=x, k_out=x)


def test_a_cache_of_the_host_is_refused():
    with pytest.raises(ValueError, match="CUDA"):
        KvCache(4, 2, 64, 16, "int8", device="cpu")
    pages = torch.zeros((4, 2, 1, 1, 16, 64), dtype=torch.int8)
    with pytest.raises(ValueError, match="CUDA"):
        KvCache(4, 2, 64, 16, "int8", k_pages=pages)


class Where:
    """A tensor, as far as KvCache looks at one, of a device that need not be there."""

    def __init__(self, device, shape, dtype):
        self.device, self.shape, self.dtype = torch.device(device), torch.Size(shape), dtype

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 0x10000


def test_the_four_buffers_of_a_cache_are_of_one_device():
    def buffers(*devices):
        return {name: Where(d, shape, dt) for name, d, shape, dt in zip(
            ("k_pages", "v_pages", "k_scales", "v_scales"), devices,
            ((4, 2, 1, 1, 16, 64), (4, 2, 1, 16, 4, 4, 4), (4, 2), (4, 2)),
            (torch.int8, torch.int8, torch.float32, torch.float32))}

    KvCache(4, 2, 64, 16, "int8", **buffers("cuda:0", "cuda:0", "cuda:0", "cuda:0"))
    KvCache(4, 2, 64, 16, "int8", device="cuda", **buffers("cuda:1", "cuda:1", "cuda:1", "cuda:1"))
    for i in range(1, 4):
        devices = ["cuda:0"] * 4
        devices[i] = "cuda:1"
        with pytest.raises(ValueError, match="cuda:0"):
            KvCache(4, 2, 64, 16, "int8", **buffers(*devices))
    with pytest.raises(ValueError):
        KvCache(4, 2, 64, 16, "int8", device="cuda:1", **buffers(*["cuda:0"] * 4))


class Stream:
    def __init__(self, device):
        self.device = torch.device(device)


def test_a_stream_of_another_device_is_refused():
    """(Such a call used to run again without the stream.)"""
    ran = []
    with pytest.raises(ValueError, match="cuda:1"):
        attention._elsewhere(lambda *a, **kw: ran.append(1), 0, Stream("cuda:1"), ())
    assert not ran


def test_growth_of_a_cache_is_checked():
    import ctypes

    from adapter_gemm_linear_gb300 import _lib, build
    build()
    with pytest.raises(ValueError, match="growth"):
        KvCache(4, 2, 64, 16, "int8", growth="most")
    # the field lies where the structure had four unused bytes
    assert _lib.KvCacheDesc.growth.offset == 20 and _lib.KvCacheDesc.k_pages.offset == 24 and ctypes.sizeof(_lib.KvCacheDesc) == 56
    heads, batch = _lib.Heads(None, 256, 128), _lib.KvBatch(0, 0, None, None, None, 1)
    for growth, status in ((0, "LORA_OK"), (1, "LORA_OK"), (2, "LORA_ERR_UNSUPPORTED"), (-1, "LORA_ERR_UNSUPPORTED")):
        desc = _lib.KvCacheDesc(0, 4, 2, 128, 16, growth, 0x10000, 0x10000, 0x10000, 0x10000)
        got = _lib.lib().lora_kv_append(ctypes.byref(desc), ctypes.byref(batch), 0, ctypes.byref(heads), ctypes.byref(heads), None)
        assert got == _lib.STATUS[status]
