"""CPU tier: the host code of the linears over an 8-bit base and of the draw of
tokens under AddressSanitizer and UndefinedBehaviorSanitizer: their sources and the C ABI's
(device code unchanged), with tests/int8_asan_driver.cpp.  The launchers of
the other entries are not linked; the driver calls none of them."""
import concurrent.futures as cf
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"
SOURCES = ["tenant_fine_tune_amd/csrc/api.cpp", "tenant_fine_tune_amd/csrc/quantize.hip",
           "tenant_fine_tune_amd/csrc/linear_int8.hip", "tenant_fine_tune_amd/csrc/linear_int8_tiles.hip",
           "tenant_fine_tune_amd/csrc/sample.hip", "tenant_fine_tune_amd/csrc/gemm.hip", "tests/int8_asan_driver.cpp"]


def test_int8_and_sample_host_code_under_asan_and_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-omit-frame-pointer", "-Xarch_host", "-fno-sanitize-recover=undefined"]

    def comp(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([HIPCC, "-O1", "-g", "-std=c++17", "-fPIC", "-x", "hip", "--offload-arch=gfx950", *san,
                            "-I", os.path.join(ROOT, "include"), "-c", os.path.join(ROOT, src), "-o", obj],
                           capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-3000:]
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(6, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(comp, SOURCES))
    exe = str(tmp_path / "int8_driver")
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", *san, "-Wl,--unresolved-symbols=ignore-all", *objs, "-o", exe],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    env = {**os.environ, "ASAN_OPTIONS": "detect_leaks=0:abort_on_error=0:halt_on_error=1",
           "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1"}
    run = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    out = run.stdout + run.stderr
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert run.returncode == 0, out[-4000:]
    assert "int8 driver: 0 failures" in run.stdout
