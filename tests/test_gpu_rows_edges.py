"""GPU: edges of the router's, the expert MLP's and the adapter linear's range.

Definitions, checks and tolerances are those of test_gpu_rows.py.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_rows import (check_lora, check_moe, codes, gen, lora_case, moe_case, moe_ref, pack, randn,  # noqa: E402
                           w4)  # noqa: F401

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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("top", [1e-30, 5e-37, 3.6e-37, 1e-37, 1e-38])
@pytest.mark.parametrize("M,K", [(1, 256), (4, 3584), (40, 1152), (3, 40960)])
def test_codes_of_tiny_rows(w4, M, K, top, dtype):  # noqa: F811
    """Rows so small that 1 / (absmax / 127) overflows float32 have the codes of the rule all the same."""
    g = gen(M + K)
    x = (randn(g, M, K).double() * (top / 8)).clamp(-top, top).to(dtype)
    x[:, 7], x[:, 9] = 0.0, top
    qa, sa = w4.quant_act(x)
    c, s = codes(x)
    assert torch.equal(sa.double(), s)
    assert torch.equal(qa.double(), c)


@pytest.mark.parametrize("M,k,E", [(1, 4, 6), (40, 2, 8), (60, 4, 3), (3000, 3, 3)])
def test_moe_of_tiny_intermediate_rows(w4, M, k, E):  # noqa: F811
    """silu(gate) * up of about 1e-37, brought back to the normal range by the down weight."""
    k = min(k, E)
    x, up, down, ids, wt = moe_case(M, M, k, E, 640, 1280, torch.bfloat16)
    up, down = (up[0], up[1], up[2] * 2.0 ** -63), (down[0], down[1], down[2] * 2.0 ** 40)
    y = w4.moe_mlp(x, *pack(w4, up, down, E), ids, wt)
    ref, slack = moe_ref(x, up, down, ids, wt, E)
    assert 0 < float(ref.abs().max()) < 1e-20
    check_moe(y.double() * 2.0 ** 80, ref * 2.0 ** 80, slack * 2.0 ** 80)


@pytest.mark.parametrize("M", [1, 8, 40, 300])
def test_lora_of_tiny_rows(w4, M):  # noqa: F811
    """The shared product of such rows, beside which the adapters' is nothing."""
    x, w, A, B, sc, ids = lora_case(M, M, 1152, 528, 3, 16, torch.float32)
    x = x * 2.0 ** -130
    w = (w[0], w[1], w[2] * 2.0 ** 40)
    check_lora(w4.lora_linear(x, w4.pack_weights(*w), w4.LoraAdapters(A, B, sc), ids), x, w, A, B, sc, ids)


@pytest.mark.parametrize("M,K,N,L,R", [((1 << 20) + 300, 128, 32, 3, 8), (113152 + 300, 18944, 32, 4, 16)])
def test_lora_passes(w4, M, K, N, L, R):  # noqa: F811
    """More rows than one pass takes, by their number and by the 2^31 bytes of
    their codes: rows before, at and after the border against the definition."""
    p = w4.lora_linear_plan(M, N, K, L, R)
    assert p.rows == M - 300
    g = gen(M)
    block = randn(g, 4099, K)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, M, 4099):
        x[lo: lo + 4099] = block[: min(4099, M - lo)]
    _, w, A, B, sc, _ = lora_case(7, 1, K, N, L, R, torch.bfloat16)
    ids = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    y = w4.lora_linear(x, w4.pack_weights(*w), w4.LoraAdapters(A, B, sc), ids)
    for lo in (0, M - 400, M - 200):
        r = slice(lo, lo + 200)
        check_lora(y[r], x[r], w, A, B, sc, ids[r])


def test_moe_passes_by_bytes(w4):  # noqa: F811
    """A pass ends where a token's codes would pass 2^31 bytes."""
    k, E, I, K = 1, 4, 128, 18944
    M = (2 ** 31 - 1) // K + 150
    assert w4.moe_mlp_plan(M, k, E, I, K).tokens == M - 150
    x, up, down, _, _ = moe_case(5, 2, k, E, I, K, torch.bfloat16)
    g = gen(6)
    block = randn(g, 4099, K)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, M, 4099):
        x[lo: lo + 4099] = block[: min(4099, M - lo)]
    ids = torch.randint(-1, E, (M, k), generator=g, device="cuda", dtype=torch.int32)
    wt = torch.rand(M, k, generator=g, device="cuda")
    y = w4.moe_mlp(x, *pack(w4, up, down, E), ids, wt)
    for lo in (0, M - 250, M - 100):
        r = slice(lo, lo + 100)
        check_moe(y[r], *moe_ref(x[r], up, down, ids[r], wt[r], E))


@pytest.mark.parametrize("M", [1, 20, 70])
def test_moe_most_experts_and_slots(w4, M):  # noqa: F811
    x, up, down, ids, wt = moe_case(M, M, 64, 1024, 128, 128, torch.float32, drop=0.1)
    y = w4.moe_mlp(x, *pack(w4, up, down, 1024), ids, wt)
    check_moe(y, *moe_ref(x, up, down, ids, wt, 1024))
