"""CPU: the size limits that include/w4a8_mx.h states are those that the calls have,
on both sides of each."""
import ctypes

import pytest

from test_mx_abi_cpu import INVALID, SHAPE, _grouped, _linear, lib  # noqa: F401

LIMIT = 1 << 32


def plan(lib, M, N, K, act, E=0):  # noqa: F811
    from bit_quantized_amd import _lib
    p = _lib.MxPlan()
    rc = lib.w4a8_mx_grouped_linear_plan(M, M, E, N, K, act, ctypes.byref(p)) if E else \
        lib.w4a8_mx_linear_plan(M, N, K, act, ctypes.byref(p))
    return rc, p


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("M", [1, 4, 33, 300])
@pytest.mark.parametrize("K", [32, 128, 160, 256, 512, 2048, 2912, 8192, 1 << 22])
def test_channels_times_inputs(lib, M, K, act):  # noqa: F811
    """N times K rounded up to 128 below 2^32: odd and even numbers of steps of 128 alike."""
    most = (LIMIT - 1) // (-(-K // 128) * 128) // 16 * 16
    for N, ok in ((most, True), (most + 16, False)):
        assert (plan(lib, M, N, K, act)[0] == 0) == ok
        assert (plan(lib, M, N, K, act, E=1)[0] == 0) == ok
        assert bool(lib.w4a8_mx_linear_workspace_bytes(M, N, K, act)) == ok
        status = INVALID if ok else SHAPE  # (a call without its output)
        assert _linear(lib, M=M, N=N, K=K, act=act, y=None) == status
        assert _grouped(lib, M=M, P=M, E=1, N=N, K=K, act=act, y=None) == status


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("M,E", [(1 << 24, 0), ((1 << 24) - 77, 0), (1 << 24, 1), (1 << 24, 1000), (1 << 14, 1024)])
def test_threads_of_a_launch(lib, M, E, act):  # noqa: F811
    """The most channels that M rows take are those of the stated launch."""
    K = 32
    lo, hi = 1, (1 << 31) // max(E, 1) // 16  # in 16 channels
    hi = min(hi, LIMIT // 128 // 16 - 1)
    assert plan(lib, M, 16 * lo, K, act, E)[0] == 0
    refused, _ = plan(lib, M, 16 * hi, K, act, E)
    if refused == 0:
        pytest.skip("every weight of these sizes can be launched")
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if plan(lib, M, 16 * mid, K, act, E)[0] == 0 else (lo, mid)
    _, p = plan(lib, M, 16 * lo, K, act, E)
    assert p.path == 3 and plan(lib, M, 16 * hi, K, act, E)[0] == SHAPE
    tiles = -(-M // p.tile_rows) + min(E, M)
    assert tiles * -(-16 * lo // p.tile_cols) * 512 < LIMIT
    assert tiles * -(-16 * hi // p.tile_cols) * 512 >= LIMIT
