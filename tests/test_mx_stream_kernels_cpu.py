"""CPU: the microscaled streams that are built are those that a plan of the GPU
tests' sizes takes, and no others."""
import os
import re
import subprocess

import pytest

pytest.importorskip("torch")

import bit_quantized_amd as w4  # noqa: E402
import test_gpu_mx as products  # noqa: E402
import test_gpu_mx_supers as supers  # noqa: E402


def built(tmp_path):
    from bit_quantized_amd import build as B
    out = str(tmp_path / "mx_stream.s")
    r = subprocess.run([B.HIPCC, *B.FLAGS, "--cuda-device-only", "-S", os.path.join(B.CSRC, "mx_stream.hip"), "-o",
                        out], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    with open(out) as f:
        names = re.findall(r"^\s*\.amdhsa_kernel (\S+)", f.read(), re.M)
    found = {tuple(map(int, re.search(r"ILi(\d)ELi(\d)ELi(\d)ELi(\d)ELb(\d)E", n).groups())) for n in names}
    assert len(found) == len(names)
    return found


def taken():
    """(format, row tiles, raw type, channel blocks, gated) of every plan of the tests."""
    out = set()
    for f, act in enumerate(products.FMTS):
        plans = [(w4.mx_linear_plan(*s, act), False) for s in products.LINEAR]
        plans += [(w4.mx_linear_plan(*s[:3], act), False) for s in supers.LINEAR[act]]
        plans += [(w4.mx_grouped_linear_plan(37, sum(c) + 7, len(c), N, K, act), g)
                  for c, N, K, g in products.grouped_sizes()]
        for p, gated in plans:
            if p.path == w4.MX_TILE:
                continue
            blocks = 2 if gated else p.tile_cols // 16
            for raw in (1, 2) if p.path == w4.MX_TOKEN else (0,):  # bfloat16 and float rows
                out.add((f, p.tile_rows // 16, raw, blocks, int(gated)))
    return out


def test_every_stream_that_is_built_is_taken(tmp_path):
    assert built(tmp_path) == taken()
