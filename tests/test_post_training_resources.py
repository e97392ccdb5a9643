"""The post-training kernels at compile time, on the CPU: none needs scratch
memory (a spill inside their loops costs more than anything they gain), and the
tile kernels leave room for the workgroups per compute unit that their launch
rules count on."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "packed_quantized_lm_amd", "csrc")
LDS = 160 * 1024


@pytest.fixture(scope="module")
def usage():
    from packed_quantized_lm_amd import build as b
    hipcc = os.path.join(b.ROCM, "bin", "hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    runs = [subprocess.Popen([hipcc, *b.HIP_FLAGS, f"-I{b.INCLUDE}", f"-I{CSRC}", os.path.join(CSRC, src),
                              "--cuda-device-only", "-c", "-o", os.devnull, "-Rpass-analysis=kernel-resource-usage"],
                             stdout=subprocess.DEVNULL, stderr=subprocess.PIPE, text=True)
            for src in ("loss.hip", "fp8.hip", "backward.hip")]
    found, name = {}, None
    for p in runs:
        err = p.communicate()[1]
        assert p.returncode == 0, err[-2000:]
        for line in err.splitlines():
            m = re.search(r"Function Name: (\S+)", line)
            if m:
                name = m.group(1)
                found[name] = {}
            m = re.search(r"remark: +([A-Za-z ]+?)(?: \[[^\]]*\])?: (\d+)", line)
            if m and name:
                found[name][m.group(1).strip()] = int(m.group(2))
    return found


def test_no_kernel_needs_scratch_memory(usage):
    assert len(usage) > 40
    for n, u in usage.items():
        assert u.get("ScratchSize", -1) == 0, f"{n} spills: {u}"


@pytest.mark.parametrize("kernel,count,groups", [
    ("11tile_kernelILi32E", 1, 3), ("11tile_kernelILi64E", 1, 2), ("11tile_kernelILi256E", 1, 1),
    ("product_tile_kernelILi64ELi128E", 2, 3), ("product_tile_kernelILi128ELi128E", 2, 2)])
def test_workgroups_per_compute_unit(usage, kernel, count, groups):
    found = {n: u for n, u in usage.items() if kernel in n}
    assert len(found) == count, sorted(usage)
    for n, u in found.items():
        waves = 4 if "ELi128E" in kernel and "product" in kernel else 8
        assert u["LDS Size"] * groups <= LDS and u["Occupancy"] * 4 >= groups * waves, f"{n}: {u}"
