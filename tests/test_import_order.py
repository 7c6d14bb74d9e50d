"""CPU tier: one HIP runtime a process, whichever of torch and the package is
imported first (with two, torch's and the system's, the library finds no
device)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("order", ["torch, tenant_fine_tune_amd", "tenant_fine_tune_amd, torch"])
def test_one_hip_runtime(order):
    code = (f"import {order}\n"
            "print(len({line.split()[-1] for line in open('/proc/self/maps') if 'libamdhip64' in line}))")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split()[-1] == "1"
