"""A rule of the norms' source that no run can show broken (no GPU needed)."""

import re

from test_attention_source import source


def test_the_ring_begins_at_a_multiple_of_the_pieces_that_change_places():
    """Interleaved, a thread's two 16-byte pieces are 32 bytes of which the second is found by an exclusive or with 16: the
    dynamic shared memory has to be declared at a multiple of 32."""
    text = source("attn_norm_rope.cu")
    assert re.search(r"chunk \^ 16u", text)
    declared = re.findall(r"extern __shared__ __align__\((\d+)\) unsigned char smem\[\];", text)
    assert len(declared) == 2 == len(re.findall(r"extern __shared__", text)) and all(int(n) % 32 == 0 for n in declared)
