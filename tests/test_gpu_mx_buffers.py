"""GPU: the microscaled operators on buffers as a program may hold them: at the least
alignment, in one workspace that two captured graphs share."""
import pytest

torch = pytest.importorskip("torch")

import mx_reference as ref  # noqa: E402
from test_gpu_mx import FMTS, gen, w4, weight  # noqa: E402,F401

pytestmark = pytest.mark.gpu

LINEAR = [(1, 256, 672), (16, 4112, 2080), (40, 256, 1056), (33, 256, 9248), (150, 4112, 288), (300, 18960, 416),
          (1030, 12816, 288)]
GROUPS = [((1, 0, 2, 1), 64, 1056), ((4, 0, 9, 1, 6, 0, 0, 3), 96, 2080), ((70, 3, 90), 288, 544),
          ((300, 250, 500), 352, 800)]


def shifted(t):
    """A copy that begins 16 bytes past a 256-byte line."""
    raw = torch.empty(t.numel() * t.element_size() + 512, dtype=torch.uint8, device="cuda")
    at = -raw.data_ptr() % 256 + 16
    out = raw[at:at + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 256 == 16
    return out


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("size", LINEAR, ids=str)
def test_linear_at_the_least_alignment(w4, act, size):  # noqa: F811
    M, N, K = size
    g = gen(M)
    q, s = weight(g, N, K)
    w = w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda())
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).cuda()
    want = w4.mx_linear(x, w, act=act)
    moved = w4.mx_pack_weights(shifted(ref.pack4(q).cuda()), shifted(s.cuda()), out=shifted(torch.zeros_like(w.buf)))
    assert torch.equal(moved.buf, w.buf)
    ws = shifted(torch.zeros(w4.mx_linear_workspace_bytes(M, N, K, act), dtype=torch.uint8))
    y = w4.mx_linear(shifted(x), moved, act=act, out=shifted(torch.zeros_like(want)), workspace=ws)
    assert torch.equal(y, want)
    t, u = w4.mx_quant(x, act), w4.mx_quant(shifted(x), act)
    u = w4.MxTensor(shifted(u.codes), shifted(u.scales), act)
    assert torch.equal(t.codes, u.codes) and torch.equal(t.scales, u.scales)
    assert torch.equal(w4.mx_dequant(u, out=shifted(torch.zeros_like(x))), w4.mx_dequant(t))


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("case", GROUPS, ids=lambda c: f"{sum(c[0])}rows")
def test_groups_at_the_least_alignment(w4, act, gated, case):  # noqa: F811
    counts, N, K = case
    E, P, M = len(counts), sum(counts), 37
    g = gen(P)
    q, s = weight(g, E * N, K)
    w = w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda(), n_experts=E)
    x = torch.randn(M, K, generator=g).cuda()
    rows = torch.randint(0, M, (P,), generator=g, dtype=torch.int32).cuda()
    offsets = torch.cumsum(torch.tensor([0] + list(counts)), 0).to(torch.int32).cuda()
    want = w4.mx_grouped_linear(x, w, offsets, rows=rows, gated=gated, act=act)
    ws = shifted(torch.zeros(w4.mx_grouped_linear_workspace_bytes(M, P, E, N, K, act), dtype=torch.uint8))
    y = w4.mx_grouped_linear(shifted(x), w4.MxWeight(shifted(w.buf), E, N, K), shifted(offsets), rows=shifted(rows),
                             gated=gated, act=act, out=shifted(torch.zeros_like(want)), workspace=ws)
    assert torch.equal(y, want)


def captured(call):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    return graph


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("rows", [(9, 40), (33, 150)])
def test_two_graphs_share_a_workspace(w4, act, rows):  # noqa: F811
    """A linear and a grouped product, captured apart, replayed in turn and interleaved with eager
    calls in the same workspace: whatever one leaves there does not show in the other."""
    g = gen(sum(rows))
    N, K, E = 4112, 2080, 4
    counts = [rows[1] // 2, 0, rows[1] - rows[1] // 2, 0]
    (q, s), (qs, ss) = weight(g, N, K), weight(g, E * 96, K)
    one = w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda())
    all_ = w4.mx_pack_weights(ref.pack4(qs).cuda(), ss.cuda(), n_experts=E)
    a = torch.randn(rows[0], K, generator=g).to(torch.bfloat16).cuda()
    b = torch.randn(rows[1], K, generator=g).to(torch.bfloat16).cuda()
    offsets = torch.cumsum(torch.tensor([0] + counts), 0).to(torch.int32).cuda()
    ws = torch.empty(max(w4.mx_linear_workspace_bytes(rows[0], N, K, act),
                         w4.mx_grouped_linear_workspace_bytes(rows[1], rows[1], E, 96, K, act)),
                     dtype=torch.uint8, device="cuda")
    ya = torch.empty(rows[0], N, dtype=torch.bfloat16, device="cuda")
    yb = torch.empty(rows[1], 96, dtype=torch.bfloat16, device="cuda")
    ga = captured(lambda: w4.mx_linear(a, one, act=act, out=ya, workspace=ws))
    gb = captured(lambda: w4.mx_grouped_linear(b, all_, offsets, act=act, out=yb, workspace=ws))
    for i in range(4):
        a.copy_(torch.randn(a.shape, generator=gen(i)))
        b.copy_(torch.randn(b.shape, generator=gen(10 + i)))
        ya.zero_()
        yb.zero_()
        for graph in ((ga, gb, ga), (gb, ga, gb))[i % 2]:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ya, w4.mx_linear(a, one, act=act, workspace=ws)), f"linear, replay {i}"
        assert torch.equal(yb, w4.mx_grouped_linear(b, all_, offsets, act=act, workspace=ws)), f"groups, replay {i}"
