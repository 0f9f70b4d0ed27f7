"""GPU: streams of microscaled weights whose wavefronts share several runs of 512
inputs: every number of row tiles, one and two channel blocks a workgroup, the
last run not full, and runs enough that a wavefront takes more than one.

Definitions are those of test_gpu_mx.py, the comparison that of mx_strict.py.
"""
import pytest

pytest.importorskip("torch")

import mx_strict  # noqa: E402
import test_gpu_mx as products  # noqa: E402
from test_gpu_mx import FMTS, w4  # noqa: E402,F401

pytestmark = pytest.mark.gpu

# (rows, channels, inputs, channels of a workgroup) of the linear, by the rows' format
LINEAR = {
    "fp4": [(16, 4112, 8160, 16), (20, 4112, 8160, 16), (40, 4096, 8160, 16), (64, 4112, 4064, 16),
            (20, 8208, 2080, 32), (20, 8208, 8160, 32), (48, 8208, 2080, 32), (47, 8208, 7904, 32),
            (64, 8192, 2048, 32), (60, 8208, 5152, 32)],
    "fp8": [(16, 4112, 8160, 16), (20, 4112, 4064, 16), (40, 4096, 4064, 16), (64, 4096, 4064, 16),
            (20, 8208, 2080, 32), (20, 8208, 4832, 32), (48, 8208, 2080, 32), (47, 8208, 3168, 32),
            (64, 8208, 640, 32), (60, 8192, 608, 32)],
}
# (rows of each group, channels, inputs); an odd number of 16-channel blocks too
GROUPED = [((3, 0, 8, 1, 16, 9, 5, 9), 48, 2912), ((8, 6, 7, 0, 9, 6), 96, 9248), ((1, 2, 0, 20, 3), 1056, 8544)]


@pytest.fixture(autouse=True)
def strict(monkeypatch):
    monkeypatch.setattr(products, "check", mx_strict.check)


@pytest.mark.parametrize("act,size", [(a, s) for a in FMTS for s in LINEAR[a]], ids=str)
def test_linear_streamed_over_several_runs(w4, act, size):  # noqa: F811
    M, N, K, cols = size
    p = w4.mx_linear_plan(M, N, K, act)
    assert (p.path, p.tile_rows, p.tile_cols) == (w4.MX_STREAM, -(-M // 16) * 16, cols)
    for near in (True, False):
        products.linear_case(w4, M, N, K, act, "floor", "bf16", near)


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("case", GROUPED, ids=lambda c: f"{sum(c[0])}rows_{c[1]}x{c[2]}")
def test_groups_streamed_over_several_runs(w4, act, case):  # noqa: F811
    counts, N, K = case
    for tail in (0, 7):
        assert w4.mx_grouped_linear_plan(37, sum(counts) + tail, len(counts), N, K, act).path == w4.MX_STREAM
    products.grouped_case(w4, counts, N, K, act, tail=7)
    products.grouped_case(w4, counts, N, K, act, gather=False, dtype="f32", rule="ceil", near=False)
    if N % 32 == 0:
        products.grouped_case(w4, counts, N, K, act, gated=True, tail=7)
