"""CPU tier: how an attention call's work is cut from device-side lengths
(csrc/attention_schedule.h), walked on the host over hundreds of random
batches, with and without values that make no sense: every key weighed once,
every partial state written before it is read, every index inside its array."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"


def test_schedule_covers_and_bounds(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "schedule_check")
    r = subprocess.run([HIPCC, "-O1", "-std=c++17", "-x", "hip", "--offload-arch=gfx950", "-D_GLIBCXX_ASSERTIONS",
                        "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=undefined",
                        os.path.join(ROOT, "tests", "schedule_check.cpp"), "-o", exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "schedule: 0 failures" in run.stdout, run.stdout + run.stderr
