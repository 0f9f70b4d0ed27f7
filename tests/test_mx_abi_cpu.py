"""CPU: include/w4a8_mx.h without a GPU.  Every refusal returns its status on the
host, before anything is enqueued; a workspace serves every smaller number of
rows; the GPU tests' sizes reach every kernel that a plan can take."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_amd import _lib
    return _lib.load()


def P(v):
    return ctypes.c_void_p(v)


BASE = 1 << 40      # aligned addresses far apart, never dereferenced
STEP = 1 << 38


def _ptr(i):
    return P(BASE + i * STEP)


MIS = P(BASE + 4)
INVALID, SHAPE, MISALIGNED, SMALL = -1, -2, -3, -4


def _quant(lib, x=_ptr(0), dtype=0, M=4, K=96, fmt=0, rule=0, codes=_ptr(1), scales=_ptr(2)):
    return lib.w4a8_mx_quant(x, dtype, M, K, fmt, rule, codes, scales, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INVALID), (dict(M=-1), INVALID), (dict(M=(1 << 24) + 1), INVALID), (dict(K=0), INVALID),
    (dict(K=-32), INVALID), (dict(K=40), SHAPE), (dict(K=16), SHAPE), (dict(K=(1 << 22) + 32), SHAPE),
    (dict(dtype=2), INVALID), (dict(fmt=2), INVALID), (dict(fmt=-1), INVALID), (dict(rule=2), INVALID),
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(x=MIS), MISALIGNED),
    (dict(codes=MIS), MISALIGNED), (dict(scales=MIS), MISALIGNED), (dict(codes=_ptr(0)), INVALID),
    (dict(scales=_ptr(0)), INVALID), (dict(scales=_ptr(1)), INVALID), (dict(scales=P(BASE + STEP + 176)), INVALID),
])
def test_quant_refusals(lib, kw, status):
    assert _quant(lib, **kw) == status
    assert lib.w4a8_last_error() != b""


def _dequant(lib, codes=_ptr(0), scales=_ptr(1), fmt=0, M=4, K=96, y=_ptr(2), dtype=0):
    return lib.w4a8_mx_dequant(codes, scales, fmt, M, K, y, dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INVALID), (dict(K=33), SHAPE), (dict(dtype=5), INVALID), (dict(fmt=7), INVALID),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(y=None), INVALID), (dict(y=MIS), MISALIGNED),
    (dict(codes=MIS), MISALIGNED), (dict(y=_ptr(0)), INVALID), (dict(y=_ptr(1)), INVALID),
])
def test_dequant_refusals(lib, kw, status):
    assert _dequant(lib, **kw) == status
    assert lib.w4a8_last_error() != b""


def _pack(lib, codes=_ptr(0), scales=_ptr(1), N=32, K=96, packed=_ptr(2), pb=1 << 30):
    return lib.w4a8_mx_pack_weights(codes, scales, N, K, packed, pb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), INVALID), (dict(N=24), SHAPE), (dict(N=(1 << 31) + 16), INVALID), (dict(K=0), INVALID),
    (dict(K=48), SHAPE), (dict(K=(1 << 22) + 32), SHAPE), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(packed=None), INVALID), (dict(pb=64), SMALL), (dict(codes=MIS), MISALIGNED), (dict(packed=MIS), MISALIGNED),
    (dict(packed=_ptr(0)), INVALID), (dict(packed=_ptr(1)), INVALID),
])
def test_pack_refusals(lib, kw, status):
    assert _pack(lib, **kw) == status
    assert lib.w4a8_last_error() != b""
    kw = dict(kw)
    if "pb" in kw or not {"codes", "scales", "packed"} & set(kw):
        a = dict(N=32, K=96, pb=1 << 30)
        a.update(kw)
        assert lib.w4a8_mx_unpack_weights(_ptr(2), a["pb"], a["N"], a["K"], _ptr(0), _ptr(1), None) == status


@pytest.mark.parametrize("N,K", [(16, 32), (16, 128), (48, 160), (32, 544), (64, 3584), (80, 2912), (16, 1 << 22)])
def test_weight_bytes_match_the_layout(lib, N, K):
    G, Q = -(-K // 128) | 1, -(-K // 512) | 1
    need = N // 16 * (G * 1024 + Q * 256) + 1024
    assert lib.w4a8_mx_weight_bytes(N, K) == need
    assert _pack(lib, N=N, K=K, pb=need - 1) == SMALL
    assert lib.w4a8_mx_weight_bytes(N, K + 16) == 0 and lib.w4a8_mx_weight_bytes(N + 8, K) == 0


def _linear(lib, x=_ptr(0), dtype=0, act=0, rule=0, packed=_ptr(1), pb=1 << 40, M=4, N=64, K=96, y=_ptr(2),
            ws=_ptr(3), wsb=1 << 36):
    return lib.w4a8_mx_linear(x, dtype, act, rule, packed, pb, M, N, K, y, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INVALID), (dict(M=(1 << 24) + 1), INVALID), (dict(N=0), INVALID), (dict(N=40), SHAPE),
    (dict(K=0), INVALID), (dict(K=100), SHAPE), (dict(N=1 << 22, K=1 << 12), SHAPE), (dict(dtype=2), INVALID),
    (dict(act=2), INVALID), (dict(act=-1), INVALID), (dict(rule=2), INVALID), (dict(x=None), INVALID),
    (dict(packed=None), INVALID), (dict(y=None), INVALID), (dict(ws=None), SMALL), (dict(wsb=64), SMALL),
    (dict(pb=64), SMALL), (dict(x=MIS), MISALIGNED), (dict(packed=MIS), MISALIGNED), (dict(y=MIS), MISALIGNED),
    (dict(ws=MIS), MISALIGNED), (dict(y=_ptr(0)), INVALID), (dict(ws=_ptr(0)), INVALID), (dict(ws=_ptr(1)), INVALID),
    (dict(y=_ptr(3)), INVALID), (dict(M=1 << 24, N=1 << 24, K=32), SHAPE),
])
def test_linear_refusals(lib, kw, status):
    assert _linear(lib, **kw) == status
    assert lib.w4a8_last_error() != b""


def _grouped(lib, x=_ptr(0), dtype=0, act=0, rule=0, packed=_ptr(1), pb=1 << 40, offsets=_ptr(2), rows=_ptr(3),
             M=4, P=40, E=8, N=64, K=96, gated=0, y=_ptr(4), ws=_ptr(5), wsb=1 << 36):
    return lib.w4a8_mx_grouped_linear(x, dtype, act, rule, packed, pb, offsets, rows, M, P, E, N, K, gated, y, ws,
                                      wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), INVALID), (dict(P=0), INVALID), (dict(P=(1 << 24) + 1), INVALID), (dict(E=0), INVALID),
    (dict(E=1025), INVALID), (dict(N=40), SHAPE), (dict(N=48, gated=1), SHAPE), (dict(K=100), SHAPE),
    (dict(N=1 << 22, K=1 << 12), SHAPE), (dict(E=1024, N=1 << 22), INVALID), (dict(dtype=2), INVALID),
    (dict(act=2), INVALID), (dict(rule=-1), INVALID), (dict(rows=None), INVALID), (dict(x=None), INVALID),
    (dict(packed=None), INVALID), (dict(offsets=None), INVALID), (dict(y=None), INVALID), (dict(ws=None), SMALL),
    (dict(wsb=64, P=400), SMALL), (dict(pb=64), SMALL), (dict(x=MIS), MISALIGNED), (dict(offsets=MIS), MISALIGNED),
    (dict(rows=MIS), MISALIGNED), (dict(y=MIS), MISALIGNED), (dict(ws=MIS), MISALIGNED), (dict(y=_ptr(0)), INVALID),
    (dict(y=_ptr(2)), INVALID), (dict(y=_ptr(3)), INVALID), (dict(ws=_ptr(2)), INVALID), (dict(y=_ptr(5)), INVALID),
    (dict(M=1 << 20, K=1 << 13), SHAPE),     # rows by index past 32-bit offsets
    (dict(P=1 << 24, N=1 << 20, K=32), SHAPE),
])
def test_grouped_refusals(lib, kw, status):
    assert _grouped(lib, **kw) == status
    assert lib.w4a8_last_error() != b""


def test_buffer_edges(lib):
    """One byte short of each documented size is refused; the documented size is not (the call then
    lacks its output)."""
    need = lib.w4a8_mx_weight_bytes(64, 96)
    assert _linear(lib, pb=need - 1) == SMALL and _linear(lib, pb=need, y=None) == INVALID
    need = lib.w4a8_mx_weight_bytes(8 * 64, 96)
    assert _grouped(lib, pb=need - 1) == SMALL and _grouped(lib, pb=need, y=None) == INVALID
    # y ends where the workspace begins, or a byte past it
    M, N = 4, 64
    assert _linear(lib, y=P(BASE + 3 * STEP - M * N * 2), M=M, N=N, x=None) == INVALID
    assert b"null" in lib.w4a8_last_error()
    assert _linear(lib, y=P(BASE + 3 * STEP - M * N * 2 + 16), M=M, N=N) == INVALID
    assert b"alias" in lib.w4a8_last_error()


def fewer(M):
    """Row counts up to M: all of the small ones, the edges of the tiles, a spread of the rest."""
    some = set(range(1, min(M, 530) + 1)) | {M}
    for t in range(64, M + 1, 64):
        some |= {t - 1, t, min(t + 1, M)}
    v = 1.0
    while v < M:
        some.add(int(v))
        v *= 1.07
    return sorted(some)


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("N,K", [(18944, 3584), (3584, 18944), (3584, 3584), (256, 384), (16, 32), (16, 65536),
                                 (65536, 256), (1040, 131072), (4112, 2912)])
def test_linear_workspace_serves_fewer_rows(lib, N, K, act):
    for M in (2, 16, 17, 64, 65, 256, 257, 2048, 9000):
        have = lib.w4a8_mx_linear_workspace_bytes(M, N, K, act)
        assert have
        for m in fewer(M):
            got = _linear(lib, M=m, N=N, K=K, act=act, wsb=have, y=None)
            assert got == INVALID, f"{m} rows: status {got}, {have} bytes asked for {M}"
    ask = [lib.w4a8_mx_linear_workspace_bytes(m, N, K, act) for m in fewer(9000)]
    assert all(a <= b for a, b in zip(ask, ask[1:]))


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("E,N,K", [(128, 1536, 2048), (8, 256, 384), (1, 64, 32), (1024, 32, 64), (64, 2560, 3584)])
def test_grouped_workspace_serves_fewer_rows(lib, E, N, K, act):
    for M, most in ((1, 16), (64, 600), (4096, 30000), (30000, 30000)):
        have = lib.w4a8_mx_grouped_linear_workspace_bytes(M, most, E, N, K, act)
        assert have
        for p in fewer(most):
            for m in {1, min(M, p), M}:
                got = _grouped(lib, M=m, P=p, E=E, N=N, K=K, act=act, wsb=have, y=None)
                assert got == INVALID, f"{m}, {p} rows: status {got}, {have} bytes asked for {M}, {most}"


# what the GPU tests of linear and grouped products must reach: (kernel, rows, columns, split)
def test_gpu_tests_reach_every_kernel(lib):
    pytest.importorskip("torch")
    import bit_quantized_amd as w4
    import test_gpu_mx as gpu
    for act in gpu.FMTS:
        plans = [w4.mx_linear_plan(M, N, K, act) for M, N, K in gpu.LINEAR]
        seen = {(p.path, p.tile_rows, p.tile_cols, p.ksplit > 1) for p in plans}
        want = {(w4.MX_TOKEN, 16, 16, False)}
        want |= {(w4.MX_STREAM, 16, 16, False)} | {(w4.MX_STREAM, r, c, False) for r in (32, 48, 64) for c in (16, 32)}
        want |= {(w4.MX_TILE, *t, s) for t in ((64, 128), (128, 128), (128, 256), (256, 256)) for s in (False, True)}
        assert want <= seen, want - seen
        grouped = [(w4.mx_grouped_linear_plan(37, sum(c) + 7, len(c), N, K, act), gated)
                   for c, N, K, gated in gpu.grouped_sizes()]
        seen = {(p.path, p.tile_rows, p.tile_cols, g) for p, g in grouped}
        want = {(w4.MX_TOKEN, 16, 16, g) for g in (False, True)} | {(w4.MX_STREAM, 16, 32, g) for g in (False, True)}
        want |= {(w4.MX_TILE, *t, g) for t in ((64, 128), (128, 128), (128, 256), (256, 256)) for g in (False, True)}
        assert want <= seen, want - seen


def test_plan_queries_refuse(lib):
    from bit_quantized_amd import _lib
    plan = _lib.MxPlan()
    assert lib.w4a8_mx_linear_plan(4, 64, 96, 0, None) == INVALID
    assert lib.w4a8_mx_grouped_linear_plan(4, 8, 2, 64, 96, 0, None) == INVALID
    for a, status in (((0, 64, 96, 0), INVALID), ((4, 40, 96, 0), SHAPE), ((4, 64, 96, 3), INVALID)):
        assert lib.w4a8_mx_linear_plan(*a, ctypes.byref(plan)) == status
        assert lib.w4a8_mx_linear_workspace_bytes(*a) == 0
    for a, status in (((4, 0, 2, 64, 96, 0), INVALID), ((4, 8, 2, 64, 100, 0), SHAPE)):
        assert lib.w4a8_mx_grouped_linear_plan(*a, ctypes.byref(plan)) == status
        assert lib.w4a8_mx_grouped_linear_workspace_bytes(*a) == 0


def test_python_refusals():
    """The binding's own checks, on CPU tensors: nothing reaches the library."""
    torch = pytest.importorskip("torch")
    import bit_quantized_amd as w4
    x, u8 = torch.zeros(2, 64), torch.zeros(32, 32, dtype=torch.uint8)
    with pytest.raises(ValueError):
        w4.mx_quant(x)                                       # not on the GPU
    with pytest.raises(ValueError):
        w4.mx_quant(x, "fp6")
    with pytest.raises(ValueError):
        w4.mx_quant(x, rule="nearest")
    with pytest.raises(ValueError):
        w4.mx_dequant(w4.MxTensor(u8, torch.zeros(32, 1, dtype=torch.uint8), "fp4"))  # 64 values, one scale
    with pytest.raises(TypeError):
        w4.mx_dequant(w4.MxTensor(u8.int(), torch.zeros(32, 2, dtype=torch.uint8), "fp4"))
    with pytest.raises(ValueError):
        w4.mx_pack_weights(u8, torch.zeros(32, 2, dtype=torch.uint8))  # not on the GPU
    with pytest.raises(ValueError):
        w4.mx_linear(x, w4.MxWeight(u8, 1, 32, 64))
    with pytest.raises(ValueError):
        w4.mx_grouped_linear(x, w4.MxWeight(u8, 2, 16, 64), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        w4.mx_linear_workspace_bytes(4, 64, 96, "int8")
    with pytest.raises(w4._lib.W4A8Error):
        w4.mx_linear_plan(4, 40, 96)
