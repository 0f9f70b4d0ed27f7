"""GPU: the microscaled operators as a program uses them: together, captured and
replayed, on several streams, in the least workspace, past 32-bit offsets.

Definitions, checks and tolerances are those of test_gpu_mx.py.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mx_reference as ref  # noqa: E402
from test_gpu_mx import FMTS, activations, check, gen, w4, weight  # noqa: E402,F401


def pack(w4, q, s, n_experts=1):  # noqa: F811
    return w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda(), n_experts=n_experts)


def by_expert(ids, E):
    """The pairs of ids [M][k] in expert order: their rows, the experts' offsets, and the order."""
    flat = ids.reshape(-1).long()
    flat = torch.where((flat < 0) | (flat >= E), E, flat)
    order = torch.sort(flat, stable=True).indices
    # (no histogram: a comparison and a sum, which a graph replays)
    counts = (flat[:, None] == torch.arange(E, device=ids.device)).sum(dim=0)
    ends = torch.cumsum(counts, 0)
    offsets = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
    return (order // ids.shape[1]).to(torch.int32), offsets, order


class Layer:
    """A router and the experts' gated MLP on 4-bit microscaled weights."""

    def __init__(self, w4, E, K, I, act, seed):  # noqa: F811
        g = gen(seed)
        self.w4, self.E, self.act = w4, E, act
        self.router = torch.randn(E, K, generator=g).cuda() / K ** 0.5
        self.qu, self.qd = weight(g, E * 2 * I, K), weight(g, E * K, I)
        self.up, self.down = pack(w4, *self.qu, n_experts=E), pack(w4, *self.qd, n_experts=E)

    def step(self, x, k, parts=None):
        scores = x.float() @ self.router.t()
        ids, weights = self.w4.moe_route(scores, k)
        rows, offsets, order = by_expert(ids, self.E)
        h = self.w4.mx_grouped_linear(x, self.up, offsets, rows=rows, gated=True, act=self.act)
        y = self.w4.mx_grouped_linear(h, self.down, offsets, act=self.act)
        out = torch.empty_like(y)
        out[order] = y  # the pairs in the tokens' order
        if parts is not None:
            parts.update(ids=ids, offsets=offsets, rows=rows, h=h, y=y)
        M, K = x.shape
        return (out.view(M, k, K).float() * weights[:, :, None]).sum(dim=1).to(torch.bfloat16)


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_router_and_experts_together(w4, act, M):  # noqa: F811
    """Every product of the step against its definition on the inputs that it had."""
    E, K, inter, k = 8, 288, 160, 3
    layer = Layer(w4, E, K, inter, act, M)
    x = activations(gen(M), M, K, True).to(torch.bfloat16).cuda()
    p = {}
    got = layer.step(x, k, p)
    off = p["offsets"].tolist()
    assert off[-1] == M * k and bool(torch.isfinite(got).all())
    xv, hv = ref.rounded(x, act, "floor"), ref.rounded(p["h"], act, "floor")
    wu, wd = (ref.values(q.cuda(), s.cuda(), "fp4") for q, s in (layer.qu, layer.qd))
    for e in range(E):
        run = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        rows = p["rows"][run].long()
        assert bool((p["ids"][rows] == e).any(dim=1).all())
        we = wu[e * 2 * inter:(e + 1) * 2 * inter]
        v, (err, cut) = xv[rows] @ we.t().contiguous(), ref.slack(xv[rows], we, act)
        gate, val, half = v[:, :inter], v[:, inter:], inter
        err = 1.1 * err[:, :half] * val.abs() + gate.abs() * err[:, half:] + 1.1 * err[:, :half] * err[:, half:]
        check(p["h"][run], ref.silu_mul(v), err + ref.silu_mul(v).abs() * 2.0 ** -20, f"up {e}")
        we = wd[e * K:(e + 1) * K]
        err, cut = ref.slack(hv[run], we, act)
        check(p["y"][run], hv[run] @ we.t().contiguous(), err + cut, f"down {e}")


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("M", [1, 6, 70])
def test_captured_step(w4, act, M):  # noqa: F811
    """The whole step as a graph, replayed with new tokens, eager work between the replays."""
    layer = Layer(w4, 8, 288, 160, act, 3)
    x = torch.randn(M, 288, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x, 3)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.step(x, 3)
    for i in range(4):
        x.copy_(torch.randn(M, 288, generator=gen(i)))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, layer.step(x, 3)), f"replay {i}"


LINEAR = [(1, 256, 672), (3, 64, 4096), (16, 272, 1056), (40, 256, 1056), (33, 256, 9248), (100, 4112, 672),
          (300, 2064, 800), (700, 144, 4128)]


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear_captured_and_in_other_workspaces(w4, act, M, N, K):  # noqa: F811
    """The same bits captured and replayed, in a workspace of more rows, in the least one that a call
    takes (nothing is written behind it), whatever it holds, and again."""
    g = gen(M + N)
    w = pack(w4, *weight(g, N, K))
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).cuda()
    y0 = w4.mx_linear(x, w, act=act)
    assert torch.equal(w4.mx_linear(x, w, act=act), y0)
    more = torch.full((w4.mx_linear_workspace_bytes(M + 500, N, K, act),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(w4.mx_linear(x, w, act=act, workspace=more), y0)
    from test_mx_abi_cpu import _linear
    lib, lo, hi = w4.load(), 0, w4.mx_linear_workspace_bytes(M, N, K, act)
    while hi - lo > 1:  # lo is too small, hi is not: found by calls without an output
        mid = (lo + hi) // 2
        status = _linear(lib, M=M, N=N, K=K, act=FMTS.index(act), wsb=mid, y=None)
        assert status in (-4, -1)
        lo, hi = (mid, hi) if status == -4 else (lo, mid)
    buf = torch.randint(0, 256, (hi + 4096,), device="cuda", dtype=torch.uint8)
    tail = buf[hi:].clone()
    out = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    w4.mx_linear(x, w, act=act, workspace=buf[:hi], out=out[:M])
    assert torch.equal(out[:M], y0) and torch.equal(buf[hi:], tail) and bool((out[M:] == 7.0).all())
    ws = torch.empty(hi, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w4.mx_linear(x, w, act=act, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph, y = torch.cuda.CUDAGraph(), torch.empty_like(y0)
    with torch.cuda.graph(graph):
        w4.mx_linear(x, w, act=act, workspace=ws, out=y)
    for i in range(3):
        x.copy_(torch.randn(M, K, generator=gen(i)))
        ws.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, w4.mx_linear(x, w, act=act)), f"replay {i}"


@pytest.mark.parametrize("act", FMTS)
def test_two_streams_at_once(w4, act):  # noqa: F811
    """Calls with workspaces of their own on two streams at the same time."""
    g = gen(5)
    cases = [(200, 2064, 800), (9, 4112, 672)]
    ws = [pack(w4, *weight(g, N, K)) for _, N, K in cases]
    xs = [torch.randn(M, K, generator=g).to(torch.bfloat16).cuda() for M, _, K in cases]
    want = [w4.mx_linear(x, w, act=act) for x, w in zip(xs, ws)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(w4.mx_linear(xs[i], ws[i], act=act))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(y, want[i]) for y in got[i])


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("E,P", [(3, 12), (40, 60), (3, 100), (3, 400), (2, 1600)])
def test_offsets_that_do_not_ascend_stay_inside(w4, act, E, P):  # noqa: F811
    """Offsets past the rows, negative or falling are bounded: rows that only sound groups name are
    right, nothing outside y is written, and rows of no group stay as they were."""
    K, N = 160, 64
    g = gen(E)
    x = activations(g, P, K, True).to(torch.bfloat16).cuda()
    q, s = weight(g, E * N, K)
    w = pack(w4, q, s, n_experts=E)
    big = 2 ** 31 - 1
    xv, wv = ref.rounded(x, act, "floor"), ref.values(q.cuda(), s.cuda(), "fp4")
    first = P // 2
    for rest in ([big] * E, [-5] * E, [0, big] * E, [first, -big - 1, big] * E):
        offsets = torch.tensor([0, first] + rest, dtype=torch.int64)[:E + 1].to(torch.int32)
        buf = torch.full((P + 64, N), 7.5, dtype=torch.bfloat16, device="cuda")
        y = buf[32:32 + P]
        w4.mx_grouped_linear(x, w, offsets.cuda(), act=act, out=y)
        torch.cuda.synchronize()
        assert bool((buf[:32] == 7.5).all()) and bool((buf[32 + P:] == 7.5).all())
        sound = all(r >= first or r < 0 for r in offsets[2:].tolist()) and -5 in rest
        if sound:  # group 0 alone has rows
            e, _ = ref.slack(xv[:first], wv[:N], act)
            check(y[:first], xv[:first] @ wv[:N].t().contiguous(), e, f"{offsets.tolist()}")
            assert bool((y[first:] == 7.5).all())


def test_a_row_does_not_depend_on_the_others(w4):  # noqa: F811
    """Under one plan: other rows beside it, another place in the batch."""
    g = gen(1)
    for M, N, K in ((16, 272, 1056), (48, 256, 544), (100, 272, 672), (300, 2064, 544)):
        w = pack(w4, *weight(g, N, K))
        x = torch.randn(M, K, generator=g).to(torch.bfloat16).cuda()
        for act in FMTS:
            y = w4.mx_linear(x, w, act=act)
            turned = w4.mx_linear(x.flip(0).contiguous(), w, act=act)
            assert torch.equal(turned.flip(0), y)
            other = torch.randn(M, K, generator=g).to(torch.bfloat16).cuda()
            other[M // 2] = x[M // 2]
            assert torch.equal(w4.mx_linear(other, w, act=act)[M // 2], y[M // 2])


# --------------------------------------------------- past 32-bit offsets

def test_more_rows_than_one_launch_quantises(w4):  # noqa: F811
    """8.5 million rows: their quantisation takes two launches, their codes pass 2^30 bytes."""
    M, N, K = (1 << 23) + 100001, 16, 32
    g = gen(2)
    q, s = weight(g, N, K)
    w = pack(w4, q, s)
    some = torch.randn(4099, K, generator=g).to(torch.bfloat16).cuda()
    x = some.repeat(-(-M // 4099), 1)[:M].contiguous()
    y = w4.mx_linear(x, w)
    want = w4.mx_linear(some, w)
    xv, wv = ref.rounded(some, "fp4", "floor"), ref.values(q.cuda(), s.cuda(), "fp4")
    check(want, xv @ wv.t().contiguous(), ref.slack(xv, wv, "fp4")[0])
    for at in (0, (1 << 23) // 4099 * 4099, (M - 1) // 4099 * 4099):
        n = min(4099, M - at)
        assert torch.equal(y[at:at + n], want[:n]), f"rows from {at}"


def test_quantising_past_2_to_32_values(w4):  # noqa: F811
    """9.1e9 values: two launches each way, codes past 2^32 bytes."""
    M, K = 1 << 24, 544
    some = torch.randn(4096, K, generator=gen(3)).to(torch.bfloat16).cuda()
    x = some.repeat(M // 4096, 1)
    t = w4.mx_quant(x)
    want = w4.mx_quant(some)
    edge = (1 << 33) // K // 4096 * 4096  # the rows around the second launch's first value
    for at in (0, edge, M - 4096):
        assert torch.equal(t.codes[at:at + 4096], want.codes) and torch.equal(t.scales[at:at + 4096], want.scales)
    back, values = w4.mx_dequant(t, out=x), w4.mx_dequant(want)
    for at in (0, edge, M - 4096):
        assert torch.equal(back[at:at + 4096], values), f"rows from {at}"


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("counts", [{0: 3, 63: 5}, {0: 40, 62: 500, 63: 700}])
def test_experts_past_2_to_32_bytes(w4, act, counts):  # noqa: F811
    """64 experts of 16384 x 8192 weights: 4.6e9 bytes, the last ones past 32-bit offsets."""
    E, N, K = 64, 16384, 8192
    g = torch.Generator(device="cuda").manual_seed(4)
    codes = torch.randint(0, 256, (E * N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(118, 122, (E * N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    w = w4.mx_pack_weights(codes, scales, n_experts=E)
    assert w.buf.numel() > 1 << 32
    back = w4.mx_unpack_weights(w)
    assert torch.equal(back.codes, codes) and torch.equal(back.scales, scales)
    P = sum(counts.values())
    per = torch.zeros(E, dtype=torch.int64)
    for e, n in counts.items():
        per[e] = n
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(per, 0)]).to(torch.int32)
    x = activations(gen(6), P, K, True).to(torch.bfloat16).cuda()
    y = w4.mx_grouped_linear(x, w, offsets.cuda(), act=act)
    xv = ref.rounded(x, act, "floor")
    for e in counts:
        run = slice(int(offsets[e]), int(offsets[e + 1]))
        for rows in (slice(e * N, e * N + 512), slice((e + 1) * N - 512, (e + 1) * N)):
            wv = ref.values(ref.unpack4(codes[rows]), scales[rows], "fp4")
            err, _ = ref.slack(xv[run], wv, act)
            cols = slice(rows.start - e * N, rows.stop - e * N)
            check(y[run, cols], xv[run] @ wv.t().contiguous(), err, f"expert {e}")


def test_packing_past_2_to_32_pieces(w4):  # noqa: F811
    """68.9e9 bytes of codes: more pieces of 16 bytes than one launch has threads."""
    K, some = 8192, 4096
    N = (1 << 36) // (K // 2) + some
    g = gen(9)
    part = torch.randint(0, 256, (some, K // 2), generator=g, dtype=torch.uint8).cuda()
    part_s = torch.randint(0, 255, (some, K // 32), generator=g, dtype=torch.uint8).cuda()
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((N, K // 32), dtype=torch.uint8, device="cuda")
    codes.view(-1, some, K // 2)[:] = part
    scales.view(-1, some, K // 32)[:] = part_s
    w, want = w4.mx_pack_weights(codes, scales), w4.mx_pack_weights(part, part_s).buf
    stride, per = (K // 128 + 1) * 1024, (K // 512 + 1) * 256  # of 16 channels; both counts made odd
    plane = N // 16 * stride
    n, m = some // 16 * stride, some // 16 * per
    for at in (0, N // some // 2, N // some - 1):
        assert torch.equal(w.buf[at * n:(at + 1) * n], want[:n]), at
        assert torch.equal(w.buf[plane + at * m:plane + (at + 1) * m], want[n:n + m]), at
    codes.zero_()
    scales.zero_()
    del codes, scales
    back = w4.mx_unpack_weights(w)
    for at in (0, N // some // 2, N // some - 1):
        assert torch.equal(back.codes[at * some:(at + 1) * some], part), at
        assert torch.equal(back.scales[at * some:(at + 1) * some], part_s), at
    del w, back
    torch.cuda.empty_cache()


@pytest.mark.parametrize("act", FMTS)
def test_outputs_past_2_to_32_bytes(w4, act):  # noqa: F811
    """2^20 rows of 4112 outputs, linear and by expert with rows read by index."""
    M, N, K, E = 1 << 20, 4112, 96, 2
    x = activations(gen(12), 4096, K, True).to(torch.bfloat16).cuda()
    q, s = weight(gen(13), E * N, K)
    w = pack(w4, q, s, n_experts=E)
    xv, wv = ref.rounded(x, act, "floor"), ref.values(q.cuda(), s.cuda(), "fp4")
    cut = M // 2 + 1000
    offsets = torch.tensor([0, cut, M], dtype=torch.int32).cuda()
    rows = torch.arange(M, dtype=torch.int32).cuda() % 4096
    one = w4.MxWeight(pack(w4, q[:N], s[:N]).buf, 1, N, K)
    for whole in (True, False):
        y = w4.mx_linear(x.repeat(M // 4096, 1), one, act=act) if whole else \
            w4.mx_grouped_linear(x, w, offsets, rows=rows, act=act)
        for at in (0, cut - 300, (1 << 32) // (2 * N) - 100, M - 300):
            for lo, hi in ((at, min(at + 300, max(cut, at))), (max(at, cut), at + 300)):
                if whole:
                    lo, hi = at, at + 300
                if lo >= hi:
                    continue
                we = wv[:N] if whole or lo < cut else wv[N:]
                part = xv[rows[lo:hi].long()]
                e, _ = ref.slack(part, we, act)
                check(y[lo:hi], part @ we.t().contiguous(), e, f"rows from {lo}")
        del y
