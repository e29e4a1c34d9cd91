"""The generated gfx950 code of the weight-gradient kernels of large tiles.

Its loop waits for copies into LDS that the compiler does not know of, by
counting the memory instructions issued since: the wait lets 2 loads per chunk
of X and the copies of one stage stay in flight. Fewer instructions between two
waits than that would let a stage start on data that has not arrived; a spill in
the loop would add others and slow it down. Compiled here without a GPU."""

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
    out = tmp_path_factory.mktemp("asm") / "wgrad.s"
    cmd = [HIPCC, "-O3", "-std=c++17", "--offload-arch=gfx950", "--cuda-device-only", "-S",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", os.path.join(CSRC, "wgrad_kernels.hip"), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = out.read_text().split("\n")
    found = {}
    for i, l in enumerate(lines):
        m = re.match(r"^(_ZN4muon\d+wgrad_kernelILi(\d)EEEv\S*):", l)
        if m:
            end = next(j for j in range(i, len(lines)) if "s_endpgm" in lines[j])
            found[int(m.group(2))] = [x.strip() for x in lines[i:end]]
    assert sorted(found) == [0, 1], "one kernel for each element type"
    return found


VMEM = re.compile(r"^(global|buffer|scratch|flat)_(load|store|atomic)")


@pytest.mark.parametrize("kind", [0, 1])
def test_the_wait_never_allows_more_than_was_issued_since(kernels, kind):
    body = kernels[kind]
    waits = [i for i, l in enumerate(body) if re.match(r"s_waitcnt vmcnt\(\d+\) lgkmcnt\(0\)", l) and "s_barrier" in "".join(body[i:i + 2])]
    assert len(waits) == 3, "two stages in the loop and an odd last one"
    counts = []
    for i in waits:
        allowed = int(re.search(r"vmcnt\((\d+)\)", body[i]).group(1))
        # straight back through this stage's 26 MFMAs before the meeting
        issued = mfma = 0
        for l in reversed(body[:i]):
            if l.startswith("v_mfma"):
                mfma += 1
                if mfma > 26:
                    break
            issued += bool(VMEM.match(l))
        counts.append((issued, allowed))
    # The odd last stage is followed by none: its loads of X are dropped, and
    # what its wait would be for is not read.
    assert all(issued >= allowed for issued, allowed in counts[:2]), counts


@pytest.mark.parametrize("kind", [0, 1])
def test_no_spills(kernels, kind):
    assert not [l for l in kernels[kind] if l.startswith("scratch_")]


# The kernel of 128 x 128 tiles is the same loop with 16 MFMAs a stage.
@pytest.fixture(scope="module")
def medium(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("asm") / "wgrad.s"
    cmd = [HIPCC, "-O3", "-std=c++17", "--offload-arch=gfx950", "--cuda-device-only", "-S",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", os.path.join(CSRC, "wgrad_kernels.hip"), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = out.read_text().split("\n")
    found = {}
    for i, l in enumerate(lines):
        m = re.match(r"^(_ZN4muon\d+wgrad_medium_kernelILi(\d)EEEv\S*):", l)
        if m:
            end = next(j for j in range(i, len(lines)) if "s_endpgm" in lines[j])
            found[int(m.group(2))] = [x.strip() for x in lines[i:end]]
    assert sorted(found) == [0, 1], "one kernel for each element type"
    return found


@pytest.mark.parametrize("kind", [0, 1])
def test_medium_tiles_wait_and_keep_their_registers(medium, kind):
    body = medium[kind]
    assert not [l for l in body if l.startswith("scratch_")]
    waits = [i for i, l in enumerate(body) if re.match(r"s_waitcnt vmcnt\(\d+\) lgkmcnt\(0\)", l) and "s_barrier" in "".join(body[i:i + 2])]
    assert len(waits) == 3, "two stages in the loop and an odd last one"
    for i in waits[:2]:
        allowed = int(re.search(r"vmcnt\((\d+)\)", body[i]).group(1))
        # back to this stage's first MFMA: 12 of them go before the meeting
        issued = mfma = 0
        for l in reversed(body[:i]):
            mfma += l.startswith("v_mfma")
            if mfma > 12:
                break
            issued += bool(VMEM.match(l))
        assert issued >= allowed, (issued, allowed)
