"""GB300-native multi-adapter LoRA linear layer.

out = x W^T + per-row (alpha_i/r_i) B_i (A_i x), with adapters in a paged
pool and rows reaching them by per-row id or by sorted segments.  The work is
done by liblora.so (C ABI in include/lora.h, CUDA kernels for sm_103a); this
package only binds it to PyTorch tensors and streams.

What stands between the adapted q/k/v and o projections of a decoder layer
(include/lora_attention.h): rotary positions (rope), an 8-bit paged key/value
cache (KvCache.append, KvCache.gather) and attention over it
(KvCache.attention).
"""

from .api import (  # noqa: F401
    Int4Weight,
    Int8Weight,
    LinearCall,
    LoraError,
    LoraPool,
    abi_version,
    device_status,
    kernel_launches,
    linear_forward,
    pool_arena_bytes,
    pool_slot_bytes,
    segment_rows,
    status_string,
    arm_test_wait_timeout,
)
from .attention import KvCache, kv_pages_bytes, rope, rope_tables  # noqa: F401
from .build import build  # noqa: F401
