"""The argument checks, plans and workspace sizes of include/w4a8_rows.h under
AddressSanitizer, on the instrumented build that test_host_asan.py makes (CPU
only)."""
import os
import subprocess
import sys

import pytest

asan = pytest.importorskip("test_host_asan")

FILES = ["test_rows_abi_cpu.py", "test_rows_workspace_cpu.py", "test_rows_plan_cpu.py"]


@pytest.mark.skipif(not asan.RUNTIME, reason="no AddressSanitizer runtime in this ROCm")
def test_rows_host_checks_under_asan():
    asan._build()
    env = dict(os.environ)
    env["LD_PRELOAD"] = " ".join([asan.RUNTIME[-1]] + ([env["LD_PRELOAD"]] if env.get("LD_PRELOAD") else []))
    env["ASAN_OPTIONS"] = "detect_leaks=0:halt_on_error=1:exitcode=86"
    env["W4A8_LIB_PATH"] = asan.LIB
    probe = subprocess.run([sys.executable, "-c", "from bit_quantized_amd import _lib; print(_lib.load()._name)"],
                           cwd=asan.ROOT, env=env, capture_output=True, text=True, timeout=120)
    assert probe.returncode == 0 and probe.stdout.strip() == asan.LIB, probe.stdout + probe.stderr
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "not gpu",
                        *[os.path.join(asan.ROOT, "tests", f) for f in FILES]],
                       cwd=asan.ROOT, env=env, capture_output=True, text=True, timeout=900)
    text = r.stdout + r.stderr
    assert "AddressSanitizer" not in text, text[-4000:]
    assert r.returncode == 0, text[-4000:]
    assert " passed" in r.stdout
