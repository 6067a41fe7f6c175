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


def test_loads_from_tensor_memory_take_the_whole_warp():
    """tcgen05.ld and st are for all lanes at once: in their loops no lane goes ahead by itself, and after a wait,
    which lanes may leave apart, they meet again first."""
    text = source("attn_prefill.cu")
    softmax = text[text.index("if (warp < 8) {"):text.index("} else if (warp < 12) {")]
    for m in re.finditer(r"\bif \(([^;{}]*)\) (continue|break|return);", softmax):
        assert "rt" not in m.group(1).replace("rt_", ""), m.group(0)
    waits = [m.end() for m in re.finditer(r"wait\(&sm\.(s_full|half_done|o_done)\[X\][^;]*;", softmax)]
    assert len(waits) == 3
    for at in waits:
        assert softmax[at:].lstrip().startswith("__syncwarp();")
    store = softmax[softmax.index("for (int i = 0; i < D / 32; ++i) {"):softmax.index("part[kRows * D + rt]")]
    assert re.search(r"\}\s*__syncwarp\(\);\s*\}\s*tc_fence_before_sync", store)
