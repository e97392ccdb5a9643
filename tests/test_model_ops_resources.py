"""The kernels around the head at compile time, on the CPU: none needs scratch
memory, which would cost the bandwidth-bound ones more than anything they gain."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "packed_quantized_lm_amd", "csrc")


@pytest.mark.parametrize("source,kernels", [("norm.hip", 30), ("embed.hip", 20), ("rules.hip", 10)])
def test_no_kernel_needs_scratch_memory(source, kernels):
    from packed_quantized_lm_amd import build as b
    hipcc = os.path.join(b.ROCM, "bin", "hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    p = subprocess.run([hipcc, *b.HIP_FLAGS, f"-I{b.INCLUDE}", f"-I{CSRC}", os.path.join(CSRC, source),
                        "--cuda-device-only", "-c", "-o", os.devnull, "-Rpass-analysis=kernel-resource-usage"],
                       stdout=subprocess.DEVNULL, stderr=subprocess.PIPE, text=True)
    assert p.returncode == 0, p.stderr[-2000:]
    found, name = {}, None
    for line in p.stderr.splitlines():
        if m := re.search(r"Function Name: (\S+)", line):
            name = m.group(1)
        elif name and (m := re.search(r"ScratchSize \[bytes/lane\]: (\d+)", line)):
            found[name] = int(m.group(1))
    assert len(found) >= kernels
    assert not {n: s for n, s in found.items() if s}
