"""The weight gradient's kernel of 64 x 64 tiles hands data from lane to lane of
a wave through LDS with no workgroup barrier. The compiler knows one lane's
addresses only, so between a wave's writes and the transposing reads of what
other lanes wrote, and before the next writes, there has to be a fence. Looked
up in the compiler's gfx950 IR, without a GPU."""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_optimizer_step_muon_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("ir") / "wgrad.ll"
    cmd = [HIPCC, "-O3", "-std=c++17", "--offload-arch=gfx950", "--cuda-device-only", "-S", "-emit-llvm",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", os.path.join(CSRC, "wgrad_kernels.hip"), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    found = re.findall(r"^define [^\n]*@(_ZN4muon18wgrad_small_kernel\w+)\([^\n]*\n(.*?)^}", out.read_text(), re.M | re.S)
    assert len(found) == 4, "two element types of the checkpoint, two of dY"
    return dict(found)


def test_lds_writes_and_other_lanes_reads_are_fenced(kernels):
    for name, body in kernels.items():
        last, seen = None, 0
        for line in body.split("\n"):
            if re.search(r"\bfence\b.*wavefront|s\.barrier", line):
                last = None
            kind = "write" if re.search(r"^\s*store .*addrspace\(3\)", line) else "read" if "ds.read.tr16" in line and "call" in line else None
            if kind:
                seen += 1
                assert last in (None, kind), f"{name}: a {kind} after a {last} with nothing between them: {line.strip()}"
                last = kind
        assert seen > 20, name
