"""CPU: the GPU tests of the microscaled streams reach each of them with several
runs of 512 inputs, so with several wavefronts, and where the plan allows it
with more runs than wavefronts."""
import pytest

pytest.importorskip("torch")

import bit_quantized_amd as w4  # noqa: E402
import test_gpu_mx_supers as gpu  # noqa: E402

MOST = {16: 16, 32: 8, 48: 8, 64: 8}  # wavefronts of a workgroup, by its rows


def runs(K):
    return -(-K // 512)


@pytest.mark.parametrize("act", gpu.FMTS)
def test_every_stream_runs_over_several_wavefronts(act):
    several, more = set(), set()
    for M, N, K, cols in gpu.LINEAR[act]:
        p = w4.mx_linear_plan(M, N, K, act)
        assert (p.path, p.tile_cols) == (w4.MX_STREAM, cols)
        shape = (p.tile_rows, p.tile_cols)
        if runs(K) > 1:
            several.add(shape)
        if runs(K) > MOST[p.tile_rows]:
            more.add(shape)
    want = {(16, 16)} | {(rows, cols) for rows in (32, 48, 64) for cols in (16, 32)}
    assert several == want
    # (64 rows of 8 bits and 8192 channels go to tiles from 672 inputs on, 48 from 3232)
    assert (32, 32) in more and (act == "fp8" or {(32, 16), (48, 16), (48, 32), (64, 32)} <= more)


@pytest.mark.parametrize("act", gpu.FMTS)
def test_grouped_streams_run_over_several_wavefronts(act):
    for counts, N, K in gpu.GROUPED:
        p = w4.mx_grouped_linear_plan(37, sum(counts) + 7, len(counts), N, K, act)
        assert (p.path, p.tile_rows, p.tile_cols) == (w4.MX_STREAM, 16, 32) and runs(K) > 1
    assert any(runs(K) > MOST[16] for _, _, K in gpu.GROUPED)
    assert any(N // 16 % 2 for _, N, _ in gpu.GROUPED)
