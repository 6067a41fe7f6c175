"""The closed form of the prompt kernel's line of work (csrc/attn_sums.h), compiled for the host, against the sum itself."""

import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "adapter_gemm_linear_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "attn_sums.h"
int main() {
    for (uint32_t m = 1; m <= 64; ++m)
        for (uint32_t b = 0; b <= 200; ++b) {
            long long sum = 0;
            for (uint32_t n = 0; n <= 150; ++n) {
                if (lora::sum_of_floors(n, m, b) != sum) { std::printf("n %u m %u b %u\n", n, m, b); return 1; }
                sum += (2 * n + b) / m;
            }
        }
    for (uint32_t m = 1; m <= 64; ++m) {  // the longest sequences: 2^23 row tiles behind 2^29 / group
        const uint32_t n = (1u << 23) - 37 * m, b = (1u << 29) + 11 * m;
        long long sum = 0;
        for (uint32_t i = 0; i < n; ++i) sum += (2ull * i + b) / m;
        if (lora::sum_of_floors(n, m, b) != sum) { std::printf("large m %u\n", m); return 1; }
    }
    return 0;
}
"""


def test_sum_of_floors(tmp_path):
    (tmp_path / "sums.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "sums")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, str(tmp_path / "sums.cpp"), "-o", exe], check=True)
    done = subprocess.run([exe], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout
