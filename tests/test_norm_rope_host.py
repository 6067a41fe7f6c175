"""What lora_norm_rope and its gradient refuse on the host (no GPU needed)."""

import ctypes

import pytest
import torch

from adapter_gemm_linear_gb300 import _lib, norm_rope, norm_rope_backward
from test_attention_host import L, P, rope_args  # noqa: F401


def args(rope=None, **kw):
    a = dict(q_weight=P, k_weight=P, weight_dtype=0, unit_offset=0, eps=1e-6)
    a.update(kw)
    return _lib.NormRopeArgs(rope_args(**(rope or {})), **a)


def grads(**kw):
    a = dict(dq=_lib.Heads(P, 512, 128), dk=_lib.Heads(P, 512, 128), dq_weight=P, dk_weight=P, workspace=P, workspace_bytes=1 << 40)
    a.update(kw)
    return _lib.NormRopeGrads(**a)


@pytest.mark.parametrize("change,status", [
    (dict(rope=dict(dtype=2)), "LORA_ERR_DTYPE"), (dict(rope=dict(rows=-1)), "LORA_ERR_INVALID_ARG"),
    (dict(rope=dict(head_dim=264, q=_lib.Heads(P, 1056, 264))), "LORA_ERR_UNSUPPORTED"),
    (dict(rope=dict(inverse=1)), "LORA_ERR_UNSUPPORTED"), (dict(rope=dict(k=_lib.Heads(None, 512, 128))), "LORA_ERR_INVALID_ARG"),
    (dict(weight_dtype=2), "LORA_ERR_DTYPE"), (dict(eps=0.0), "LORA_ERR_INVALID_ARG"),
    (dict(eps=-1.0), "LORA_ERR_INVALID_ARG"), (dict(eps=float("nan")), "LORA_ERR_INVALID_ARG"),
    (dict(eps=float("inf")), "LORA_ERR_INVALID_ARG"), (dict(q_weight=P + 1), "LORA_ERR_ALIGNMENT"),
    (dict(k_weight=P + 2, weight_dtype=1), "LORA_ERR_ALIGNMENT"),
])
def test_refusals(L, change, status):  # noqa: F811
    a, g = args(**change), grads()
    assert L.lora_norm_rope(ctypes.byref(a), None) == _lib.STATUS[status]
    assert L.lora_norm_rope_backward(ctypes.byref(a), ctypes.byref(g), None) == _lib.STATUS[status]
    assert L.lora_norm_rope_backward_workspace_bytes(ctypes.byref(a)) == 0


@pytest.mark.parametrize("change,status", [
    (dict(dq=_lib.Heads(None, 512, 128)), "LORA_ERR_INVALID_ARG"), (dict(dk=_lib.Heads(P, 513, 128)), "LORA_ERR_ALIGNMENT"),
    (dict(dq_weight=P + 2), "LORA_ERR_ALIGNMENT"), (dict(workspace=None), "LORA_ERR_WORKSPACE"),
    (dict(workspace_bytes=0), "LORA_ERR_WORKSPACE"), (dict(workspace=P + 4), "LORA_ERR_ALIGNMENT"),
])
def test_refusals_of_gradients(L, change, status):  # noqa: F811
    a, g = args(), grads(**change)
    assert L.lora_norm_rope_backward(ctypes.byref(a), ctypes.byref(g), None) == _lib.STATUS[status]


def test_no_arguments_and_no_rows(L):  # noqa: F811
    bad = _lib.STATUS["LORA_ERR_INVALID_ARG"]
    assert L.lora_norm_rope(None, None) == bad and L.lora_norm_rope_backward(None, None, None) == bad
    a = args(rope=dict(rows=0))
    assert L.lora_norm_rope(ctypes.byref(a), None) == 0
    assert L.lora_norm_rope_backward(ctypes.byref(a), None, None) == bad
    g = grads(dq_weight=None, dk_weight=None, workspace=None)
    assert L.lora_norm_rope_backward(ctypes.byref(a), ctypes.byref(g), None) == 0


def test_tensors_of_the_host_are_refused():
    x = torch.zeros((2, 1, 64))
    table, pos = torch.zeros((4, 32)), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        norm_rope(x, None, None, None, table, table, pos)
    with pytest.raises(ValueError, match="CUDA"):
        norm_rope_backward(x, None, x, None, None, None, table, table, pos)
