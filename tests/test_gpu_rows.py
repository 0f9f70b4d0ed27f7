"""GPU: the router, the expert MLP and the adapter linear against plain
definitions in 64 bits.

Tolerances (fixed before the first run):
- ids are equal.  Route weights are float32: an exp of a few ulp, a sum of E
  terms and two quotients, so a relative (E + 16) 2^-24.
- lora: one rounding to bf16, 2^-8 |y|; float32 sums and operands of 16
  significant bits (x of float rows and x A^T as two bf16 parts), so 2^-14 of
  the sum of the terms' magnitudes.
- moe: one rounding to bf16, 2^-8 |y|, and h: the kernel rounds a float32
  value to bf16 where the definition rounds the 64-bit one, so an h next to a
  rounding border may differ by a step and its int8 code by one.  Per token
  four such codes are allowed for: 4 max_j(w_j hs_j) max|W_down|; over a
  whole output the error's 2-norm stays within 2^-8 + 2^-10 of the output's.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

GROUP = 128


@pytest.fixture(scope="module")
def w4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_amd as w4
    w4.load()
    return w4


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def weight(g, N, K):
    q = torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    z = torch.randint(0, 16, (N, K // GROUP), generator=g, device="cuda", dtype=torch.uint8)
    s = randn(g, N, K // GROUP).abs() * (0.2 / K ** 0.5) + 1e-4
    return q, z, s


def dequant(w):
    q, z, s = w
    N, K = q.shape
    v = (q.view(N, -1, GROUP).double() - z.double()[:, :, None]) * s.double()[:, :, None]
    return v.view(N, K)


def codes(x):
    """sa = absmax / 127 and rint(x / sa), both quotients rounded to float32 once."""
    x = x.double()
    sa = (x.abs().amax(1) / 127.0).float().double()
    t = (x / torch.where(sa == 0, 1.0, sa)[:, None]).float().double()
    return torch.round(t).clamp(-127, 127), sa


def acts(g, M, K, dtype):
    x = randn(g, M, K)
    x[:, torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]] *= 15.0
    return x.to(dtype)


# ------------------------------------------------------------------- route

def route_ref(l, k, score, bias, n_groups, topk_groups, group_top, renorm, scale):
    l = l.double().cpu()
    off = torch.isnan(l) | torch.isneginf(l)
    l = torch.where(torch.isposinf(l), torch.full_like(l, torch.finfo(torch.float32).max), l)
    l = torch.where(off, torch.full_like(l, -float("inf")), l)
    M, E = l.shape
    ids = torch.full((M, k), -1, dtype=torch.int32)
    w = torch.zeros(M, k, dtype=torch.float64)
    b = None if bias is None else bias.double().cpu()
    for m in range(M):
        on = ~off[m]
        if score == "softmax":
            p = torch.zeros(E, dtype=torch.float64)
            if on.any():
                e = torch.exp(l[m] - l[m][on].max())
                p = torch.where(on, e / e[on].sum(), 0.0)
        else:
            p = torch.where(on, torch.special.expit(l[m]), 0.0)
        c = (l[m] if b is None and (n_groups == 1 or group_top == 1) else p if b is None else p + b).tolist()
        c = [v if on[e] and v == v else -float("inf") for e, v in enumerate(c)]
        if n_groups > 1:
            per = E // n_groups
            val = []
            for gi in range(n_groups):
                best = sorted(c[gi * per:(gi + 1) * per], reverse=True)[:group_top]
                live = [v for v in best if v > -float("inf")]
                val.append(sum(live) if live else -float("inf"))
            keep = set(sorted(range(n_groups), key=lambda gi: (-val[gi], gi))[:topk_groups])
            c = [v if e // per in keep else -float("inf") for e, v in enumerate(c)]
        order = [e for e in sorted(range(E), key=lambda e: (-c[e], e)) if c[e] > -float("inf")][:k]
        for i, e in enumerate(order):
            ids[m, i], w[m, i] = e, p[e]
        if renorm:
            t = w[m].sum()
            w[m] = w[m] / t if t > 0 else 0.0
    return ids, w * scale


ROUTE = [
    # M, E, k, dtype, score, bias, n_groups, topk_groups, group_top, renorm, scale
    (1, 128, 8, "bf16", "softmax", False, 1, 1, 1, True, 1.0),
    (1, 1, 1, "f32", "softmax", False, 1, 1, 1, True, 1.0),
    (7, 61, 6, "bf16", "softmax", False, 1, 1, 1, False, 1.0),
    (130, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5),
    (33, 256, 8, "bf16", "sigmoid", True, 8, 3, 1, False, 2.5),
    (19, 96, 5, "f32", "softmax", False, 4, 2, 1, True, 1.0),
    (19, 96, 5, "bf16", "softmax", False, 4, 2, 2, True, 1.0),
    (5, 63, 9, "f32", "softmax", True, 7, 3, 2, False, 0.5),
    (9, 512, 10, "f32", "sigmoid", False, 1, 1, 1, True, 1.0),
    (6, 1024, 64, "bf16", "sigmoid", True, 64, 20, 2, True, 1.0),
    (3, 64, 64, "f32", "softmax", False, 1, 1, 1, True, 1.0),
]


@pytest.mark.parametrize("case", ROUTE, ids=lambda c: "-".join(map(str, c[:9])))
@pytest.mark.parametrize("kind", ["plain", "ties", "off", "extreme"])
def test_route(w4, case, kind):
    M, E, k, dt, score, use_bias, ng, tg, gt, renorm, scale = case
    g = gen(M * 1000 + E)
    l = randn(g, M, E) * 1.5
    if kind == "ties":
        l = torch.round(l * 2) / 2
    if kind == "off":
        l = torch.where(torch.rand(M, E, generator=g, device="cuda") < 0.6, -float("inf"), l)
        l[M // 2] = -float("inf")
        l[0, E // 2:] = float("nan")
    if kind == "extreme":
        l[0] = torch.finfo(torch.bfloat16).min
        l[M - 1, E // 2] = float("inf")
        l[M // 2, ::2] = -torch.finfo(torch.float32).max
    l = l.to(torch.bfloat16 if dt == "bf16" else torch.float32)
    bias = randn(g, E) * 0.1 if use_bias else None
    if bias is not None and kind == "ties":
        bias = torch.round(bias * 4) / 4
    ids, w = w4.moe_route(l, k, score=score, bias=bias, n_groups=ng, topk_groups=tg, group_top=gt,
                          renormalize=renorm, scale=scale)
    rid, rw = route_ref(l, k, score, bias, ng, tg, gt, renorm, scale)
    assert torch.equal(ids.cpu(), rid)
    err = (w.cpu().double() - rw).abs()
    assert torch.isfinite(w).all()
    assert (err <= (E + 16) * 2.0 ** -24 * rw.abs() + 2.0 ** -126).all(), err.max()


# --------------------------------------------------------------------- moe

def moe_ref(x, up, down, ids, weights, E):
    """(y, per-token allowance for codes next to a border), 64 bits."""
    M, K = x.shape
    inter = down[0].shape[1]
    y = torch.zeros(M, K, dtype=torch.float64, device="cuda")
    slack = torch.zeros(M, dtype=torch.float64, device="cuda")
    cx, sx = codes(x)
    for e in range(E):
        for j in range(ids.shape[1]):
            rows = torch.nonzero(ids[:, j] == e)[:, 0]
            if rows.numel() == 0:
                continue
            wu = dequant([t[e * 2 * inter:(e + 1) * 2 * inter] for t in up])
            wd = dequant([t[e * K:(e + 1) * K] for t in down])
            gu = (cx[rows] @ wu.t().contiguous()) * sx[rows][:, None]
            h = (gu[:, :inter] * torch.special.expit(gu[:, :inter]) * gu[:, inter:]).to(torch.bfloat16)
            ch, sh = codes(h)
            wt = weights[rows, j].double()
            y[rows] += wt[:, None] * sh[:, None] * (ch @ wd.t().contiguous())
            slack[rows] = torch.maximum(slack[rows], wt.abs() * sh * wd.abs().max())
    return y, 4 * slack


def moe_case(seed, M, k, E, I, K, dtype, drop=0.0, skew=False):
    g = gen(seed)
    x = acts(g, M, K, dtype)
    up, down = weight(g, E * 2 * I, K), weight(g, E * K, I)
    pref = randn(g, M, E) + (4.0 * randn(g, 1, E) if skew else 0.0)
    ids = torch.argsort(pref, dim=1, descending=True)[:, :k].to(torch.int32).contiguous()
    if drop:
        ids = torch.where(torch.rand(M, k, generator=g, device="cuda") < drop, -1, ids).contiguous()
    return x, up, down, ids, torch.softmax(randn(g, M, k), dim=1).contiguous()


def pack(w4, up, down, E):
    return w4.pack_experts(*up, n_experts=E), w4.pack_experts(*down, n_experts=E)


def check_moe(y, ref, slack):
    assert torch.isfinite(y).all()
    err = (y.double() - ref).abs()
    bound = 2.0 ** -8 * ref.abs() + slack[:, None] + 1e-30
    assert (err <= bound).all(), (err - bound).max()
    assert err.norm() <= (2.0 ** -8 + 2.0 ** -10) * ref.norm() + 1e-30


MOE = [
    # M, k, E, I, K: every tile height, and the edges between them
    (1, 1, 1, 128, 128), (1, 8, 32, 256, 512), (2, 8, 16, 128, 384), (1, 17, 20, 128, 256),
    (3, 5, 6, 384, 256), (17, 1, 3, 128, 128), (64, 4, 32, 256, 512), (5, 11, 12, 128, 640),
    (40, 4, 9, 384, 256), (100, 3, 20, 128, 384), (130, 2, 7, 256, 128), (200, 2, 8, 128, 256),
    (70, 2, 3, 640, 384), (300, 2, 4, 256, 384), (517, 3, 5, 384, 640), (257, 1, 1, 128, 256),
]


@pytest.mark.parametrize("M,k,E,I,K", MOE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_moe(w4, M, k, E, I, K, dtype):
    x, up, down, ids, wt = moe_case(M + E, M, k, E, I, K, dtype)
    y = w4.moe_mlp(x, *pack(w4, up, down, E), ids, wt)
    check_moe(y, *moe_ref(x, up, down, ids, wt, E))


@pytest.mark.parametrize("M,k,E", [(2, 4, 4), (48, 4, 16), (96, 4, 8), (300, 4, 4)])
@pytest.mark.parametrize("skew", [False, True], ids=["even", "skewed"])
def test_moe_dropped_slots(w4, M, k, E, skew):
    """Slots of experts held elsewhere (any id outside [0, E)), a token with
    none left, a weight of 0 and a zero row."""
    x, up, down, ids, wt = moe_case(7 * M, M, k, E, 256, 384, torch.bfloat16, drop=0.4, skew=skew)
    ids[M // 2] = torch.tensor([-1, E, -7, 2 ** 30], dtype=torch.int32, device="cuda")
    wt[0, 0] = 0.0
    x[M - 1] = 0.0
    y = w4.moe_mlp(x, *pack(w4, up, down, E), ids, wt)
    assert (y[M // 2] == 0).all() and (y[M - 1] == 0).all()
    check_moe(y, *moe_ref(x, up, down, ids, wt, E))


@pytest.mark.parametrize("M", [2, 20, 80, 400])
def test_moe_one_expert_for_all_and_none(w4, M):
    """All rows on the last expert, one expert twice for a token, and no row
    on any expert."""
    E = 6
    x, up, down, ids, wt = moe_case(M, M, 2, E, 128, 256, torch.float32)
    ups = pack(w4, up, down, E)
    ids[:] = E - 1
    check_moe(w4.moe_mlp(x, *ups, ids, wt), *moe_ref(x, up, down, ids, wt, E))
    ids[:] = -1
    assert (w4.moe_mlp(x, *ups, ids, wt) == 0).all()


@pytest.mark.parametrize("M,k,E,I,K", [(2, 8, 16, 128, 384), (64, 4, 32, 256, 512),
                                       (100, 3, 20, 128, 384), (300, 2, 4, 256, 384)])
def test_moe_workspace_streams_repeats(w4, M, k, E, I, K):
    """A workspace of random bytes, another stream, and repeated calls give
    the same bits; nothing past the workspace or the output is written."""
    x, up, down, ids, wt = moe_case(3, M, k, E, I, K, torch.bfloat16)
    ups = pack(w4, up, down, E)
    y0 = w4.moe_mlp(x, *ups, ids, wt)
    need = w4.moe_mlp_workspace_bytes(M, k, E, I, K)
    for seed in range(3):
        buf = torch.randint(0, 256, (need + 8192,), generator=gen(seed), device="cuda", dtype=torch.uint8)
        guard = buf.clone()
        band = torch.full((M * K + 4096,), 7.0, device="cuda", dtype=torch.bfloat16)
        out = band[2048: 2048 + M * K].view(M, K)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            w4.moe_mlp(x, *ups, ids, wt, out=out, workspace=buf[4096: 4096 + need])
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(out, y0)
        assert torch.equal(buf[:4096], guard[:4096]) and torch.equal(buf[4096 + need:], guard[4096 + need:])
        assert (band[:2048] == 7).all() and (band[2048 + M * K:] == 7).all()


def test_moe_passes(w4):
    """More pairs than one pass takes (2^19): tokens before, at and after the
    border against single-pass calls of their own."""
    k, E, I, K = 8, 4, 128, 128
    M = (1 << 16) + 300
    g = gen(5)
    x = acts(g, M, K, torch.bfloat16)
    up, down = weight(g, E * 2 * I, K), weight(g, E * K, I)
    ids = torch.randint(-1, E, (M, k), generator=g, device="cuda", dtype=torch.int32)
    wt = torch.rand(M, k, generator=g, device="cuda")
    ups = pack(w4, up, down, E)
    y = w4.moe_mlp(x, *ups, ids, wt)
    for lo in (0, (1 << 16) - 100, M - 200):
        r = slice(lo, lo + 200)
        check_moe(y[r], *moe_ref(x[r], up, down, ids[r], wt[r], E))


# -------------------------------------------------------------------- lora

def lora_case(seed, M, K, N, L, R, dtype, seg=1):
    g = gen(seed)
    x = acts(g, M, K, dtype)
    w = weight(g, N, K)
    A = (randn(g, L, R, K) / K ** 0.5).to(torch.bfloat16)
    B = (randn(g, L, N, R) / R ** 0.5).to(torch.bfloat16)
    sc = 0.25 + torch.rand(L, generator=g, device="cuda")
    ids = torch.randint(-1, L, (-(-M // seg),), generator=g, device="cuda", dtype=torch.int32)
    return x, w, A, B, sc, ids.repeat_interleave(seg)[:M].contiguous()


def check_lora(y, x, w, A, B, sc, ids):
    cx, sx = codes(x)
    dw = dequant(w)
    ref = (cx @ dw.t().contiguous()) * sx[:, None]
    mag = (cx.abs() @ dw.abs().t().contiguous()) * sx[:, None]
    for l in range(A.shape[0]):
        rows = torch.nonzero(ids == l)[:, 0]
        if rows.numel() == 0:
            continue
        a, b, s = A[l].double().t().contiguous(), B[l].double().t().contiguous(), float(sc[l])
        ref[rows] += s * ((x[rows].double() @ a) @ b)
        mag[rows] += abs(s) * ((x[rows].double().abs() @ a.abs()) @ b.abs())
    assert torch.isfinite(y).all()
    err = (y.double() - ref).abs()
    bound = 2.0 ** -8 * ref.abs() + 2.0 ** -14 * mag
    assert (err <= bound).all(), (err - bound).max()
    assert err.norm() <= 2.0 ** -8 * ref.norm()


LORA = [
    # M, K, N, L, R, seg
    (1, 128, 16, 1, 8, 1), (1, 3584, 2048, 4, 16, 1), (2, 256, 4096, 3, 24, 1), (15, 512, 272, 5, 64, 1),
    (16, 1152, 2064, 20, 128, 1), (17, 384, 528, 4, 40, 1), (33, 4736, 256, 8, 64, 1),
    (48, 640, 1040, 9, 16, 5), (64, 256, 4112, 64, 32, 1), (65, 512, 272, 3, 8, 1), (130, 1024, 784, 6, 56, 7),
    (300, 256, 4096, 12, 128, 37), (520, 384, 1296, 2, 32, 300), (1, 18944, 512, 2, 16, 1),
    (260, 4224, 256, 70, 16, 1),
]


@pytest.mark.parametrize("M,K,N,L,R,seg", LORA)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_lora(w4, M, K, N, L, R, seg, dtype):
    x, w, A, B, sc, ids = lora_case(M + N, M, K, N, L, R, dtype, seg)
    y = w4.lora_linear(x, w4.pack_weights(*w), w4.LoraAdapters(A, B, sc), ids)
    check_lora(y, x, w, A, B, sc, ids)


@pytest.mark.parametrize("M", [1, 9, 40, 90, 300])
def test_lora_ids_and_bad_adapters(w4, M):
    """Ids outside [0, L) on either side mean no adapter; an adapter that
    holds infinities and NaN reaches its own rows only."""
    K, N, L, R = 512, 784, 5, 24
    x, w, A, B, sc, ids = lora_case(M, M, K, N, L, R, torch.bfloat16)
    W = w4.pack_weights(*w)
    ids[0] = L
    if M > 2:
        ids[1], ids[2] = -(2 ** 31), 2 ** 31 - 1
    check_lora(w4.lora_linear(x, W, w4.LoraAdapters(A, B, sc), ids), x, w, A, B, sc, ids)
    B2, A2 = B.clone(), A.clone()
    B2[3, :, 1], A2[3, 2] = float("inf"), float("nan")
    y = w4.lora_linear(x, W, w4.LoraAdapters(A2, B2, sc), ids)
    keep = ids != 3
    check_lora(y[keep], x[keep], w, A, B, sc, ids[keep])
    none = torch.full_like(ids, -1)
    y = w4.lora_linear(x, W, w4.LoraAdapters(A2, B2, sc), none)
    check_lora(y, x, w, A, B, sc, none)


@pytest.mark.parametrize("M", [1, 16, 33, 300])
def test_lora_workspace_streams_repeats(w4, M):
    K, N, L, R = 1024, 2064, 6, 32
    x, w, A, B, sc, ids = lora_case(M, M, K, N, L, R, torch.float32)
    W, ad = w4.pack_weights(*w), w4.LoraAdapters(A, B, sc)
    y0 = w4.lora_linear(x, W, ad, ids)
    need = w4.lora_linear_workspace_bytes(M, N, K, L, R)
    for seed in range(3):
        buf = torch.randint(0, 256, (need + 8192,), generator=gen(seed), device="cuda", dtype=torch.uint8)
        guard = buf.clone()
        band = torch.full((M * N + 4096,), 7.0, device="cuda", dtype=torch.bfloat16)
        out = band[2048: 2048 + M * N].view(M, N)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            w4.lora_linear(x, W, ad, ids, out=out, workspace=buf[4096: 4096 + need])
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(out, y0)
        assert torch.equal(buf[:4096], guard[:4096]) and torch.equal(buf[4096 + need:], guard[4096 + need:])
        assert (band[:2048] == 7).all() and (band[2048 + M * N:] == 7).all()


# ------------------------------------------------------------------- graph

@pytest.mark.parametrize("M", [1, 24, 200])
def test_layer_in_a_graph(w4, M):
    """Router, expert MLP and adapter linear captured together, replayed with
    new inputs and eager work in between; every replay equals the eager call."""
    K, I, E, k, N, L, R = 512, 256, 8, 3, 1040, 4, 16
    g = gen(M)
    up, down, w = weight(g, E * 2 * I, K), weight(g, E * K, I), weight(g, N, K)
    ups, W = pack(w4, up, down, E), w4.pack_weights(*w)
    ad = w4.LoraAdapters((randn(g, L, R, K) / K ** 0.5).to(torch.bfloat16),
                         (randn(g, L, N, R) / R ** 0.5).to(torch.bfloat16), torch.rand(L, device="cuda"))
    x, lg = acts(g, M, K, torch.bfloat16), randn(g, M, E)
    rows = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    ws = torch.empty(max(w4.moe_mlp_workspace_bytes(M, k, E, I, K),
                         w4.lora_linear_workspace_bytes(M, N, K, L, R)), dtype=torch.uint8, device="cuda")

    def layer(x, lg, rows):
        ids, wt = w4.moe_route(lg, k)
        y = w4.moe_mlp(x, *ups, ids, wt, workspace=ws)
        return y, w4.lora_linear(y, W, ad, rows, workspace=ws)

    layer(x, lg, rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, lg, rows)
    for _ in range(4):
        x.copy_(acts(g, M, K, torch.bfloat16))
        lg.copy_(randn(g, M, E))
        rows.copy_(torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = layer(x, lg, rows)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
