"""The generated gfx950 code of the layers' products: no accumulator in memory, and
waits for the copies into LDS that leave later stages' in flight. Compiled here
without a GPU."""

import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_optimizer_step_muon_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
FILES = ("mlp_kernels", "linear8_kernels", "few_kernels")
# The largest one is fp32 in few rows with two weights: its two blocks of loads and
# their three bf16 parts need a few registers more than 16 waves leave.
SPILLS = {"few_kernelIfLi2E": 128}


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Mangled name -> (lines, bytes of scratch)."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("asm")

    def compile(name):
        cmd = [HIPCC, "-O3", "-std=c++17", "--offload-arch=gfx950", "--cuda-device-only", "-S",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", os.path.join(CSRC, name + ".hip"), "-o", str(out / (name + ".s"))]
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
        assert r.returncode == 0, r.stderr[-2000:]
        return (out / (name + ".s")).read_text()

    found = {}
    with ThreadPoolExecutor(len(FILES)) as pool:
        for text in pool.map(compile, FILES):
            for m in re.finditer(r"^(_ZN4muon\S+):.*?\n(.*?)^\s*\.end_amdhsa_kernel", text, re.M | re.S):
                scratch = int(re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", m.group(2)).group(1))
                found[m.group(1)] = [l.strip() for l in m.group(2).split("\n")], scratch
    return found


def test_what_is_kept_in_scratch(kernels):
    assert len(kernels) >= 28
    for name, (_, scratch) in kernels.items():
        allowed = next((v for k, v in SPILLS.items() if k in name), 0)
        assert scratch <= allowed, (name, scratch)


def test_a_stage_waits_for_the_copies_that_it_needs(kernels):
    """Every stage of a tile engine's loop issues its wave's copies, and meets with a
    wait that lets those of all stages but the next one stay in flight: 4 for 64 x 64
    tiles with a ring of four stages, none for a ring of two."""
    seen = 0
    for name, (body, _) in kernels.items():
        m = re.search(r"PrCfgILi(\d+)ELi\d+ELi(\d+)ELi(\d)E", name)
        if not m:
            continue
        seen += 1
        edge, row_bytes, ring = map(int, m.groups())
        per_wave = 2 * edge * row_bytes // 1024 // (8 if edge == 256 else 4)
        allowed = (ring - 2) * per_wave
        waits = [i for i, l in enumerate(body) if re.match(r"s_waitcnt vmcnt\(\d+\) lgkmcnt\(0\)", l) and body[i + 1] == "s_barrier"]
        assert waits, name
        for i in waits:
            assert int(re.search(r"vmcnt\((\d+)\)", body[i]).group(1)) <= allowed, (name, body[i])
        copies = [i for i, l in enumerate(body) if re.match(r"(global|buffer)_load\S* .*lds|global_load_lds", l)]
        assert len(copies) >= per_wave * (1 + len(waits)), (name, len(copies))
        # between two meetings a stage's copies at least
        for a, b in zip(waits, waits[1:]):
            assert sum(a < c < b for c in copies) >= per_wave, name
    assert seen == 17, "four epilogues in bf16 and the 8-bit product in three sizes, the mixed one in two"
