"""CPU-side checks of include/w4a8_rows.h: every refusal of the router, the
expert MLP and the adapter linear returns its status on the host, before
anything is enqueued (no GPU needed), and the workspaces cover what the
documented buffers take."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_amd import _lib
    return _lib.load()


def P(v):
    return ctypes.c_void_p(v)


BASE = 1 << 40      # aligned addresses far apart, never dereferenced
STEP = 1 << 36


def _ptr(i):
    return P(BASE + i * STEP)


MIS = P(BASE + 4)


def _route(lib, logits=_ptr(0), dtype=0, bias=None, M=4, E=64, k=8, score=0, n_groups=1,
           topk_groups=1, group_top=1, renorm=1, scale=1.0, ids=_ptr(1), weights=_ptr(2)):
    return lib.w4a8_moe_route(logits, dtype, bias, M, E, k, score, n_groups, topk_groups, group_top,
                              renorm, scale, ids, weights, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), -1), (dict(M=(1 << 24) + 1), -1), (dict(dtype=2), -1), (dict(E=0), -1),
    (dict(E=1025, k=1), -1), (dict(score=2), -1), (dict(score=-1), -1), (dict(k=0), -1),
    (dict(k=65, E=128), -1), (dict(E=8, k=9), -1),
    (dict(n_groups=0), -1), (dict(n_groups=7), -1), (dict(E=1024, n_groups=128), -1),
    (dict(n_groups=4, topk_groups=0), -1), (dict(n_groups=4, topk_groups=5), -1),
    (dict(n_groups=8, topk_groups=1, k=9), -1),      # a group has 8 experts
    (dict(n_groups=4, topk_groups=2, group_top=3), -1), (dict(group_top=0), -1),
    (dict(E=4, n_groups=4, topk_groups=2, group_top=2, k=1), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(logits=None), -1), (dict(ids=None), -1), (dict(weights=None), -1),
    (dict(logits=MIS), -3), (dict(bias=MIS), -3), (dict(ids=MIS), -3),
    (dict(ids=_ptr(0)), -1), (dict(weights=_ptr(1)), -1), (dict(bias=_ptr(1)), -1),
])
def test_route_refusals(lib, kw, status):
    assert _route(lib, **kw) == status
    assert lib.w4a8_last_error() != b""


def _moe(lib, x=_ptr(0), dtype=0, up=_ptr(1), down=_ptr(2), ids=_ptr(3), weights=_ptr(4), M=4, k=2,
         E=8, I=256, K=384, y=_ptr(5), ws=_ptr(6), wsb=1 << 34, upb=1 << 34, downb=1 << 34):
    return lib.w4a8_moe_mlp(x, dtype, up, upb, down, downb, ids, weights, M, k, E, I, K, y, ws, wsb,
                            None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), -1), (dict(M=(1 << 24) + 1), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(E=0), -1),
    (dict(E=1025), -1), (dict(I=0), -1), (dict(K=-128), -1), (dict(I=200), -2), (dict(K=200), -2),
    (dict(I=1 << 17, K=1 << 16), -2), (dict(dtype=3), -1),
    (dict(x=None), -1), (dict(up=None), -1), (dict(down=None), -1), (dict(ids=None), -1),
    (dict(weights=None), -1), (dict(y=None), -1), (dict(ws=None), -4), (dict(wsb=64), -4),
    (dict(upb=64), -4), (dict(downb=64), -4), (dict(x=MIS), -3), (dict(ids=MIS), -3), (dict(y=MIS), -3),
    (dict(ws=MIS), -3), (dict(y=_ptr(0)), -1), (dict(ws=_ptr(1)), -1), (dict(y=_ptr(6)), -1),
    (dict(y=_ptr(4)), -1),
])
def test_moe_refusals(lib, kw, status):
    assert _moe(lib, **kw) == status
    assert lib.w4a8_last_error() != b""


def test_moe_buffer_edges(lib):
    """One byte short of each documented size is refused."""
    M, k, E, I, K = 40, 3, 8, 256, 384
    up = lib.w4a8_packed_weight_bytes(E * 2 * I, K, 128)
    down = lib.w4a8_packed_weight_bytes(E * K, I, 128)
    ws = lib.w4a8_moe_mlp_workspace_bytes(M, k, E, I, K)
    assert ws >= M * K + M * k * (2 * I + I + 4 * K)
    a = dict(M=M, k=k, E=E, I=I, K=K)
    assert _moe(lib, upb=up - 1, **a) == -4
    assert _moe(lib, upb=up, downb=down - 1, **a) == -4
    assert _moe(lib, upb=up, downb=down, wsb=ws - 1, **a) == -4


def _lora(lib, x=_ptr(0), dtype=0, w=_ptr(1), wb=1 << 34, A=_ptr(2), B=_ptr(3), scale=_ptr(4),
          ids=_ptr(5), M=4, N=256, K=384, L=3, R=16, y=_ptr(6), ws=_ptr(7), wsb=1 << 34):
    return lib.w4a8_lora_linear(x, dtype, w, wb, A, B, scale, ids, M, N, K, L, R, y, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), -1), (dict(M=(1 << 24) + 1), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(N=250), -2),
    (dict(K=200), -2), (dict(L=0), -1), (dict(L=65537), -1), (dict(R=0), -2), (dict(R=12), -2),
    (dict(R=136), -2), (dict(N=1 << 17, K=1 << 16), -2), (dict(dtype=9), -1),
    (dict(x=None), -1), (dict(w=None), -1), (dict(A=None), -1), (dict(B=None), -1),
    (dict(scale=None), -1), (dict(ids=None), -1), (dict(y=None), -1), (dict(ws=None), -4),
    (dict(wsb=64), -4), (dict(wb=64), -4), (dict(x=MIS), -3), (dict(A=MIS), -3), (dict(B=MIS), -3),
    (dict(ids=MIS), -3), (dict(y=MIS), -3), (dict(ws=MIS), -3), (dict(y=_ptr(0)), -1),
    (dict(ws=_ptr(2)), -1), (dict(y=_ptr(7)), -1), (dict(ws=_ptr(5)), -1),
])
def test_lora_refusals(lib, kw, status):
    assert _lora(lib, **kw) == status
    assert lib.w4a8_last_error() != b""


@pytest.mark.parametrize("M", [1, 16, 17, 64, 65, 300])
def test_workspace_queries(lib, M):
    assert lib.w4a8_lora_linear_workspace_bytes(M, 256, 384, 3, 16) >= M * 384 + M * 16 * 4
    assert lib.w4a8_lora_linear_workspace_bytes(M, 250, 384, 3, 16) == 0
    assert lib.w4a8_lora_linear_workspace_bytes(M, 256, 384, 3, 7) == 0
    assert lib.w4a8_moe_mlp_workspace_bytes(M, 2, 8, 256, 384) >= M * 2 * 256 * 2
    assert lib.w4a8_moe_mlp_workspace_bytes(M, 2, 8, 250, 384) == 0
    assert lib.w4a8_moe_mlp_workspace_bytes(0, 2, 8, 256, 384) == 0


def test_workspace_of_a_long_batch_is_bounded(lib):
    """Batches whose codes pass 2^31 bytes run in passes over one workspace."""
    one = lib.w4a8_moe_mlp_workspace_bytes(1 << 16, 8, 8, 256, 4096)
    assert lib.w4a8_moe_mlp_workspace_bytes(1 << 24, 8, 8, 256, 4096) <= 16 * one
    assert lib.w4a8_lora_linear_workspace_bytes(1 << 24, 256, 384, 3, 16) < 1 << 40


def test_python_refusals():
    """The binding's own checks, on CPU tensors: nothing reaches the library."""
    torch = pytest.importorskip("torch")
    import bit_quantized_amd as w4
    with pytest.raises(ValueError):
        w4.moe_route(torch.zeros(2, 8), 2)                        # not on the GPU
    with pytest.raises(ValueError):
        w4.pack_experts(torch.zeros(30, 128, dtype=torch.uint8), None, torch.zeros(30, 1), 4)
    with pytest.raises(ValueError):
        w4.LoraAdapters(torch.zeros(1, 8, 128), torch.zeros(1, 16, 8), torch.zeros(1))
