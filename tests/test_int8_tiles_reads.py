"""CPU tier: how the tiled product over an 8-bit base reads rows that end inside 32
columns (csrc/int8_tiles.h), walked on the host: nothing past the tensor, every
number with its own column's."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"


def test_reads_stay_inside_w(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "int8_tiles_check")
    r = subprocess.run([HIPCC, "-O1", "-std=c++17", "-x", "hip", "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=undefined",
                        "-Xarch_host", "-fno-sanitize-recover=undefined", os.path.join(ROOT, "tests", "int8_tiles_check.cpp"),
                        "-o", exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "int8 tiles: 0 failures" in run.stdout, run.stdout + run.stderr
