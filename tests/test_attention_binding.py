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
