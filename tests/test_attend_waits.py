"""How long the dense attention's scheduler waits for a unit to end, worked out on the host from the kernels' own header."""

import os
import subprocess

from sparse_linear_attention_sla_b200 import build

PROGRAM = r"""
#include <cstdio>
#include "attend_common.cuh"
int main() {
  for (int bits = 0; bits <= 30; ++bits) printf("%llu\n", static_cast<unsigned long long>(sla::item_wait_ns(1 << bits)));
  printf("%llu\n", static_cast<unsigned long long>(SLA_WAIT_LIMIT_NS));
}
"""


def test_the_wait_for_a_unit_grows_with_its_steps(tmp_path):
    """The longest unit that is taken (a key tile's 2^30 query tiles) is waited for at four times the 2.1 us that a step
    was measured to take; a short one not much longer than any other wait."""
    source, binary = tmp_path / "waits.cu", tmp_path / "waits"
    source.write_text(PROGRAM)
    subprocess.run([build.nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-cudart", "static",
                    "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"), str(source), "-o", str(binary)], check=True)
    *waits, limit = map(int, subprocess.run([str(binary)], check=True, capture_output=True, text=True).stdout.split())
    for bits, ns in enumerate(waits):
        assert limit + 4 * 2100 * 2 ** bits <= ns <= limit + 10000 * 2 ** bits, bits
