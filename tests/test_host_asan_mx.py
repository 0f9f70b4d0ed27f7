"""The argument checks, plans and workspace sizes of include/w4a8_mx.h under
AddressSanitizer, on the instrumented build that test_host_asan.py makes (CPU
only)."""
import pytest

import test_host_asan_rows as rows

asan = rows.asan


@pytest.mark.skipif(not asan.RUNTIME, reason="no AddressSanitizer runtime in this ROCm")
def test_mx_host_checks_under_asan(monkeypatch):
    monkeypatch.setattr(rows, "FILES", ["test_mx_abi_cpu.py"])
    rows.test_rows_host_checks_under_asan()
