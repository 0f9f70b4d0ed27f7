"""GPU: microscaled weights of nearly 2^32 values in even numbers of steps of 128
inputs, whose odd stride brings their codes past 2^31 bytes.

Definitions are those of test_gpu_mx.py, the comparison that of mx_strict.py.
"""
import pytest

torch = pytest.importorskip("torch")

import mx_reference as ref  # noqa: E402
import mx_strict  # noqa: E402
from test_gpu_mx import FMTS, activations, gen, w4  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", params=[(16777200, 256), (2097136, 2048)], ids=str)
def wide(w4, request):  # noqa: F811
    """Packed weight, and codes and scales of some of its channels: the first and the last, and
    those around 2^31 bytes of packed codes."""
    N, K = request.param
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(119, 123, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    w = w4.mx_pack_weights(codes, scales)
    edge = (1 << 31) // ((K // 128 + 1) * 1024) * 16
    some = [(at, ref.values(ref.unpack4(codes[at:at + 256]), scales[at:at + 256], "fp4"))
            for at in (0, edge - 128, N - 256)]
    assert w.buf.numel() > 1 << 31 and edge < N - 256
    yield N, K, w, some


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("M", [1, 4, 33, 70, 200])
def test_codes_past_2_to_31_bytes(w4, wide, act, M):  # noqa: F811
    N, K, w, some = wide
    x = activations(gen(M), M, K, True).to(torch.bfloat16).cuda()
    xv = ref.rounded(x, act, "floor")
    offsets = torch.tensor([0, M], dtype=torch.int32).cuda()
    rows = torch.arange(M, dtype=torch.int32).cuda()
    calls = [lambda: w4.mx_linear(x, w, act=act),
             lambda: w4.mx_grouped_linear(x, w, offsets, rows=rows, act=act)]
    for call in calls:
        y = call()
        for at, wv in some:
            err, _ = ref.slack(xv, wv, act)
            mx_strict.check(y[:, at:at + 256], xv @ wv.t().contiguous(), err, f"channels from {at}")
        del y
