"""GPU: edges of the router's, the expert MLP's and the adapter linear's range.

Definitions, checks and tolerances are those of test_gpu_rows.py.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_rows import check_lora, lora_case, w4  # noqa: E402, F401

# between bfloat16's largest value and float32's: rounded to bfloat16 it would be an infinity
TOP = 3.4e38


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("M,K,N,seg", [(1, 512, 2064, 1), (9, 384, 272, 1), (16, 1152, 2064, 1), (40, 384, 528, 1),
                                       (90, 384, 272, 3), (1000, 256, 17424, 37)])
def test_lora_float_rows_at_the_top_of_the_range(w4, M, K, N, seg, sign):  # noqa: F811
    """Finite float rows above bfloat16's largest value, and sums x A^T above
    it, keep their adapter's product finite and within the tolerance."""
    L, R = 3, 24
    x, w, A, B, sc, ids = lora_case(M, M, K, N, L, R, torch.float32, seg)
    if M == 1:
        ids.clamp_(min=0)
    x[::2, 5] = sign * TOP
    A[:, :, 5] = 2.0 ** -7
    A[:, 3, 5] = 1.0           # the whole of it in one rank
    B = (B * 2.0 ** -10).contiguous()
    sc.fill_(1.0)
    w = (w[0], w[1], w[2] * 2.0 ** -7)
    check_lora(w4.lora_linear(x, w4.pack_weights(*w), w4.LoraAdapters(A, B, sc), ids), x, w, A, B, sc, ids)


def least_workspace(w4, M, N, K, L, R):  # noqa: F811
    """The least size a call takes: found by calls without an output, refused after that check."""
    from test_rows_abi_cpu import _lora
    lib, lo, hi = w4.load(), 0, w4.lora_linear_workspace_bytes(M, N, K, L, R)
    while hi - lo > 1:  # lo is too small, hi is not
        mid = (lo + hi) // 2
        status = _lora(lib, M=M, N=N, K=K, L=L, R=R, wsb=mid, y=None)
        assert status in (-4, -1)
        lo, hi = (mid, hi) if status == -4 else (lo, mid)
    return hi


@pytest.mark.parametrize("M", [1, 2, 16, 17, 33, 64, 65, 130, 300])
def test_lora_in_a_workspace_of_more_rows_and_in_the_least(w4, M):  # noqa: F811
    """The size asked for 300 rows serves fewer with the same bits, and a call
    writes only into the least size that it takes."""
    K, N, L, R = 1024, 2064, 6, 32
    x, w, A, B, sc, ids = lora_case(M, M, K, N, L, R, torch.bfloat16)
    W, ad = w4.pack_weights(*w), w4.LoraAdapters(A, B, sc)
    y0 = w4.lora_linear(x, W, ad, ids)
    check_lora(y0, x, w, A, B, sc, ids)
    most = torch.empty(w4.lora_linear_workspace_bytes(300, N, K, L, R), dtype=torch.uint8, device="cuda")
    assert torch.equal(w4.lora_linear(x, W, ad, ids, workspace=most), y0)
    need = least_workspace(w4, M, N, K, L, R)
    buf = torch.randint(0, 256, (need + 8192,), device="cuda", dtype=torch.uint8)
    guard = buf.clone()
    assert torch.equal(w4.lora_linear(x, W, ad, ids, workspace=buf[4096: 4096 + need]), y0)
    assert torch.equal(buf[:4096], guard[:4096]) and torch.equal(buf[4096 + need:], guard[4096 + need:])
