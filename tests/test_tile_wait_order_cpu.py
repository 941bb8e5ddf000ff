"""The 128 x 128 tile kernels start by a wait that lets stage 1's loads stay in flight
and takes stage 0's to have landed.  That holds when every copy of stage 0 is issued
before the first of the loads that it counts: checked in the assembly of the build's
own compile command, kernel by kernel (no GPU needed)."""
import os
import re
import shutil
import subprocess

import pytest

from micro_scaled_fp4_amd import build

COPIES = 8          # a wave's copies to shared memory per stage: 4 blocks of A, 4 of W


def first_wait_counts_only_later_loads(lines):
    """lines: one kernel's.  (ok, why)."""
    load = re.compile(r"^\s+(buffer|global)_load_\w+")
    points = [i for i, l in enumerate(lines) if "; order point" in l]
    if len(points) != 2:
        return False, f"{len(points)} order points"
    before = [l for l in lines[:points[0]] if load.match(l)]
    between = [l for l in lines[points[0]:points[1]] if load.match(l)]
    lds = [l for l in before if l.split(";")[0].rstrip().endswith("lds")]
    if len(lds) != COPIES:
        return False, f"{len(lds)} copies of stage 0 before the first point"
    for l in lines[points[1]:]:
        if load.match(l):
            return False, "a load between the last point and the wait"
        w = re.search(r"s_waitcnt\b.*vmcnt\((\d+)\)", l)
        if w:
            n = int(w.group(1))
            return n <= len(between), f"waits for {n} of {len(between)} later loads"
    return False, "no wait"


def test_stage_0_has_landed_at_the_first_barrier(tmp_path):
    if not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")):
        pytest.skip("no hipcc")
    out = tmp_path / "gemm_mid.s"
    subprocess.run([build._hipcc(), *build.FLAGS, "--cuda-device-only", "-S",
                    os.path.join(build.CSRC, "gemm_mid.hip"), "-o", str(out)], check=True, capture_output=True)
    kernels = re.split(r"; -- Begin function ", out.read_text())[1:]
    kernels = [k for k in kernels if k.split()[0].startswith("_ZN") and "k_gemm_mid" in k.split()[0]]
    assert len(kernels) == 16
    for k in kernels:
        ok, why = first_wait_counts_only_later_loads(k.splitlines())
        assert ok, (k.split()[0], why)


def test_the_check_finds_planted_mistakes():
    copy, plain, point = "\tbuffer_load_dwordx4 v8, s[4:7], 0 offen lds", "\tbuffer_load_dwordx2 v[2:3], v1, s[0:3], 0 offen", "\t; order point"
    wait = ["\ts_waitcnt vmcnt(9) lgkmcnt(0)", "\ts_barrier"]
    right = [plain] + [copy] * 8 + [point, plain] + [copy] * 8 + [point] + wait
    assert first_wait_counts_only_later_loads(right)[0]
    hoisted = [plain] + [copy] * 7 + [point, plain] + [copy] * 9 + [point] + wait     # a copy of stage 0 behind the point
    assert not first_wait_counts_only_later_loads(hoisted)[0]
    moved = [plain, plain] + [copy] * 8 + [point] + [copy] * 8 + [point] + wait       # the scale load before it
    assert not first_wait_counts_only_later_loads(moved)[0]
    assert not first_wait_counts_only_later_loads([l for l in right if l != point])[0]
