"""Rules of the attention kernels' source that no run can show broken (no GPU needed)."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "adapter_gemm_linear_gb300", "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def test_the_join_reads_no_fresh_data_by_the_read_only_path():
    """The joining kernel starts while the kernel before it runs: after its wait, no load that takes its data for constant."""
    text = source("attn_split.cuh")
    body = text[text.index("attn_join_kernel("):]
    before, after = body.split("griddepcontrol.wait", 1)
    after = after[:after.index("cudaError_t allow_smem")]
    assert "__ldcg" in after
    assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", before + after)
