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
