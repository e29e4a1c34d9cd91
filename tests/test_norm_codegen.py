"""The registers of the norm kernels' generated gfx950 code: the forms that rows
of up to 8192 columns (backward: 6144; aligned 8192) take keep everything in
registers. Wider ones spill, as the kernels' comments say. Compiled here without
a GPU."""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_optimizer_step_muon_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


@pytest.fixture(scope="module")
def spills(tmp_path_factory):
    """Spilled vector registers by (kernel, element type, columns / 8 per thread, aligned, most threads)."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    cmd = [HIPCC, "-O3", "-std=c++17", "--offload-arch=gfx950", "--cuda-device-only", "-S", "-Rpass-analysis=kernel-resource-usage",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", os.path.join(CSRC, "layer_kernels.hip"),
           "-o", str(tmp_path_factory.mktemp("asm") / "layer.s")]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    found = {}
    for name, rest in re.findall(r"Function Name: (\S+)(.*?)LDS Size", r.stderr, re.S):
        m = re.match(r"_ZN4muon\d+norm_(forward|backward)_kernelI([tf])Li(\d)ELb([01])E(?:Li(\d+)E)?", name)
        if m:
            kind, t, vecs, aligned, threads = m.groups()
            found[kind, {"t": "bf16", "f": "f32"}[t], int(vecs), aligned == "1", int(threads or 1024)] = int(
                re.search(r"VGPRs Spill: (\d+)", rest).group(1))
    assert len(found) == 12 + 20
    return found


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_rows_of_up_to_8192_columns(spills, dtype):
    assert spills["forward", dtype, 1, True, 1024] == 0 and spills["forward", dtype, 1, False, 1024] == 0


def test_forward_rows_of_up_to_16384_aligned_bf16_columns(spills):
    assert spills["forward", "bf16", 2, True, 1024] == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_rows_of_up_to_8192_columns(spills, dtype):
    for aligned in (True, False):
        assert spills["backward", dtype, 1, aligned, 512] == 0
    assert spills["backward", dtype, 1, True, 768] == 0 and spills["backward", dtype, 2, True, 512] == 0


def test_backward_rows_of_4097_to_6144_unaligned_columns(spills):
    assert spills["backward", "bf16", 1, False, 768] == 0
    assert spills["backward", "f32", 1, False, 768] <= 16
