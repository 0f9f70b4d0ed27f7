"""The microscaled operators (include/w4a8_mx.h) on the GPU against their
definitions in 64 bits."""
import math

import pytest
import torch

import mx_reference as ref

pytestmark = pytest.mark.gpu

FMTS = ["fp4", "fp8"]
RULES = ["floor", "ceil"]


@pytest.fixture(scope="module")
def w4():
    import bit_quantized_amd as w4
    w4.load()
    return w4


def gen(seed):
    return torch.Generator().manual_seed(seed)


def activations(g, M, K, near):
    """Normal values; near: magnitudes within a factor of 2^5, for which 8-bit products are exact."""
    x = torch.randn(M, K, generator=g)
    if near:
        x = torch.sign(x) * torch.exp2(torch.rand(M, K, generator=g) * 5 - 3)
    return x


def weight(g, N, K, mid=None):
    """Codes one a byte and scale bytes; products of order one."""
    q = torch.randint(0, 16, (N, K), generator=g, dtype=torch.uint8)
    mid = 127 - round(math.log2(2.9 * math.sqrt(K))) if mid is None else mid
    s = torch.randint(mid - 2, mid + 3, (N, K // 32), generator=g, dtype=torch.uint8)
    return q, s


def cast(x, dtype):
    return x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def same(got, want):
    """Equal values, NaN in the same places."""
    got = got.cpu()
    return got.dtype == want.dtype and bool(((got == want) | (torch.isnan(got) & torch.isnan(want))).all())


# ------------------------------------------------------------ quantisation

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 32), (1, 3584), (3, 96), (7, 2912), (65, 1056), (2, 8192 + 32)])
def test_quant_is_the_definition(w4, fmt, rule, dtype, M, K):
    g = gen(M * K)
    x = torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-40, 40, (M, K // 32), generator=g).float()
                                                    ).repeat_interleave(32, dim=1)
    x = cast(x, dtype)
    x[0, :32] = 0
    t = w4.mx_quant(x.cuda(), fmt, rule=rule)
    code, byte = ref.quantise(x, fmt, rule)
    assert torch.equal(t.scales.cpu(), byte)
    assert torch.equal(t.codes.cpu(), ref.pack4(code) if fmt == "fp4" else code)
    want = ref.values(code, byte, fmt)
    assert torch.equal(w4.mx_dequant(t, torch.float32).cpu().double(), want)
    assert torch.equal(w4.mx_dequant(t).cpu(), want.to(torch.bfloat16))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rule", RULES)
def test_quant_at_the_borders(w4, fmt, rule):
    """Every tie and its neighbours, the clipping range, the ends of the exponent range, subnormal
    and non-finite values."""
    mags = ref.magnitudes(fmt)
    ties = torch.cat([(mags[1:] + mags[:-1]) / 2, mags, torch.tensor([6.9, 7.0, 7.5, 464.0, 480.0, 511.0])])
    ties = ties[ties < 2.0 ** (ref.EMAX[fmt] + 1)].float()
    cols = torch.cat([ties, torch.nextafter(ties, ties + 1), torch.nextafter(ties, ties - 1)])
    cols = torch.cat([cols, -cols])
    top = float(mags[-1])
    rows = []
    for start in range(0, len(cols), 31):
        part = cols[start:start + 31]
        for lead in (top, 2.0 ** ref.EMAX[fmt]):
            r = torch.zeros(32)
            r[0] = lead
            r[1:1 + len(part)] = part
            rows.append(r)
    x = torch.stack(rows)
    x = torch.cat([torch.ldexp(x, torch.tensor(e)) for e in (0, -126, -133, 40, 110)])
    odd = torch.zeros(10, 32)
    odd[0, 5] = 1e-45
    odd[1, 5] = 2.0 ** -126
    odd[2, 0] = 3.3e38
    odd[3, 31] = -3.3e38
    odd[4, 7] = float("inf")
    odd[5, 8] = float("-inf")
    odd[6, 9] = float("nan")
    odd[7, :] = -0.0
    odd[8, :] = 1.2e-39
    odd[9, :2] = torch.tensor([float("nan"), 1.0])
    x = torch.cat([x, odd])
    for dtype in ("f32", "bf16"):
        xd = cast(x, dtype)
        t = w4.mx_quant(xd.cuda(), fmt, rule=rule)
        code, byte = ref.quantise(xd, fmt, rule)
        assert torch.equal(t.scales.cpu(), byte)
        assert torch.equal(t.codes.cpu(), ref.pack4(code) if fmt == "fp4" else code)
        want = ref.values(code, byte, fmt)
        for out in (torch.float32, torch.bfloat16):
            # (ceil: 4 * 2^126, past float32's largest value, is an infinity)
            assert same(w4.mx_dequant(t, out), want.to(torch.float32).to(out))


def test_dequant_of_every_code(w4):
    """All codes under scales from one end to the other, the NaN code and the NaN scale among them."""
    for fmt, n in (("fp4", 16), ("fp8", 256)):
        codes = torch.arange(n, dtype=torch.uint8).repeat(32 // 16 if n == 16 else 1).reshape(1, -1)
        for b in (0, 1, 2, 100, 127, 246, 252, 254, 255):
            scales = torch.full((1, codes.shape[1] // 32), b, dtype=torch.uint8)
            t = w4.MxTensor((ref.pack4(codes) if fmt == "fp4" else codes).cuda(), scales.cuda(), fmt)
            want = ref.values(codes, scales, fmt)
            for out in (torch.float32, torch.bfloat16):
                assert same(w4.mx_dequant(t, out), want.to(torch.float32).to(out))


@pytest.mark.parametrize("N,K", [(16, 32), (16, 128), (48, 160), (32, 544), (64, 3584), (80, 2912)])
def test_pack_round_trip_and_layout(w4, N, K):
    g = gen(N + K)
    q, s = weight(g, N, K)
    w = w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda())
    back = w4.mx_unpack_weights(w)
    assert torch.equal(back.codes.cpu(), ref.pack4(q)) and torch.equal(back.scales.cpu(), s)
    buf = w.buf.cpu()
    G, Q = -(-K // 128) | 1, -(-K // 512) | 1
    assert buf.numel() == N // 16 * (G * 1024 + Q * 256) + 1024
    full = torch.zeros(N, G * 128, dtype=torch.uint8)
    full[:, :K] = q
    want = ref.pack4(full).reshape(N // 16, 16, G, 4, 16).permute(0, 2, 3, 1, 4).reshape(-1)
    sc = torch.zeros(N, Q * 16, dtype=torch.uint8)
    sc[:, :K // 32] = s
    sc = sc.reshape(N // 16, 16, Q, 4, 4).permute(0, 2, 4, 1, 3).reshape(-1)
    assert torch.equal(buf, torch.cat([want, sc, torch.zeros(1024, dtype=torch.uint8)]))


# ----------------------------------------------------------------- products

def check(y, want, err, name=""):
    """bf16 y against 64-bit sums that float32 may miss by err, rounded once."""
    y, want = y.double().cpu(), want.cpu()
    bound = want.abs() * 2.0 ** -8 + err.cpu() * (1 + 2.0 ** -8) + 2.0 ** -133
    bad = (y - want).abs() > bound
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()}, first {torch.nonzero(bad)[0].tolist()}, " \
                          f"{y[bad][0]} against {want[bad][0]} (bound {bound[bad][0]})"


def linear_case(w4, M, N, K, act, rule, dtype, near, seed=0, **kw):
    g = gen(seed + M + 7 * N + 13 * K)
    x = cast(activations(g, M, K, near), dtype)
    q, s = weight(g, N, K)
    w = w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda())
    y = w4.mx_linear(x.cuda(), w, act=act, rule=rule, **kw)
    xv, wv = ref.rounded(x.cuda(), act, rule), ref.values(q.cuda(), s.cuda(), "fp4")
    e, cut = ref.slack(xv, wv, act)
    check(y, xv @ wv.t().contiguous(), e if near else e + cut, f"{M} {N} {K} {act}")
    return y


SIZES = [
    (1, 16, 32), (1, 48, 160), (1, 3584, 3584), (2, 64, 2912), (4, 512, 18944), (5, 256, 384), (13, 4112, 1056),
    (16, 3584, 2048), (17, 128, 32), (33, 272, 18944), (33, 3584, 4096), (64, 400, 544), (65, 4112, 2912),
    (100, 128, 128), (129, 144, 1184), (200, 2064, 640), (257, 1040, 288), (300, 16, 4096), (517, 4112, 2912)]
TILES = [
    (2048, 8192, 1056, (256, 256)), (1030, 12816, 288, (256, 256)), (300, 18960, 416, (128, 256)),
    (517, 4112, 672, (128, 128)), (200, 8208, 288, (128, 128)), (150, 4112, 288, (64, 128)), (65, 4112, 672, (64, 128))]
SLICES = [(33, 256, 18944), (100, 144, 4128), (513, 528, 16416), (70, 2064, 9248), (700, 3584, 18944),
          (130, 6544, 17472), (65, 6160, 9248), (600, 6544, 14368)]
STREAMED = [(16, 4112, 2912, 16), (17, 528, 1056, 16), (40, 4112, 544, 16), (64, 4096, 1024, 16), (20, 8208, 160, 32),
            (48, 8208, 160, 32), (60, 8208, 160, 32)]
LINEAR = SIZES + [c[:3] for c in TILES] + SLICES + [c[:3] for c in STREAMED]


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("near", [True, False])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear(w4, act, near, M, N, K):
    linear_case(w4, M, N, K, act, "floor", "bf16", near)


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 256, 672), (3, 64, 4096), (14, 128, 544), (40, 256, 1056), (150, 144, 416)])
def test_linear_of_float_rows_and_ceil(w4, act, M, N, K):
    linear_case(w4, M, N, K, act, "ceil", "f32", True)
    linear_case(w4, M, N, K, act, "floor", "f32", False)


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("M,N,K,tile", TILES)
def test_linear_of_each_tile(w4, act, M, N, K, tile):
    p = w4.mx_linear_plan(M, N, K, act)
    assert (p.path, p.tile_rows, p.tile_cols, p.ksplit) == (w4.MX_TILE, *tile, 1)
    linear_case(w4, M, N, K, act, "floor", "bf16", True)


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("M,N,K", SLICES)
def test_linear_in_slices(w4, act, M, N, K):
    assert w4.mx_linear_plan(M, N, K, act).ksplit > 1
    linear_case(w4, M, N, K, act, "floor", "bf16", True)


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("M,N,K,cols", STREAMED)
def test_linear_streamed(w4, act, M, N, K, cols):
    p = w4.mx_linear_plan(M, N, K, act)
    assert (p.path, p.tile_rows, p.tile_cols) == (w4.MX_STREAM, -(-M // 16) * 16, cols)
    linear_case(w4, M, N, K, act, "floor", "bf16", True)


def grouped_case(w4, counts, N, K, act, rule="floor", dtype="bf16", gather=True, gated=False, M=37, tail=0,
                 lead=0, near=True, seed=0, bad=()):
    E = len(counts)
    g = gen(seed + E + N + K + sum(counts))
    P = lead + sum(counts) + tail
    x = cast(activations(g, M if gather else P, K, near), dtype)
    rows = torch.randint(0, M, (P,), generator=g, dtype=torch.int32) if gather else None
    for at, v in bad:
        rows[at] = v
    offsets = torch.cumsum(torch.tensor([lead] + list(counts)), 0).to(torch.int32)
    q, s = weight(g, E * N, K)
    w = w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda(), n_experts=E)
    width = N // 2 if gated else N
    out = torch.full((P, width), 7.5, dtype=torch.bfloat16, device="cuda")
    y = w4.mx_grouped_linear(x.cuda(), w, offsets.cuda(), rows=None if rows is None else rows.cuda(), gated=gated,
                             act=act, rule=rule, out=out)
    assert y is out
    assert bool((y[:lead] == 7.5).all()) and bool((y[P - tail:] == 7.5).all())
    xv, wv = ref.rounded(x.cuda(), act, rule), ref.values(q.cuda(), s.cuda(), "fp4")
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo == hi:
            continue
        if rows is None:
            xe = xv[lo:hi]
        else:
            r = rows[lo:hi].long().cuda()
            ok = (r >= 0) & (r < M)
            xe = torch.where(ok[:, None], xv[r.clamp(0, M - 1)], 0.0)
        we = wv[e * N:(e + 1) * N]
        v = xe @ we.t().contiguous()
        e32, cut = ref.slack(xe, we, act)
        err = e32 if near else e32 + cut
        if gated:
            half = N // 2
            gate, val = v[:, :half], v[:, half:]
            # d(silu(g) u): |silu'| <= 1.1, |silu(g)| <= |g|; and float32's own rounding of the four operations
            err = 1.1 * err[:, :half] * val.abs() + gate.abs() * err[:, half:] + 1.1 * err[:, :half] * err[:, half:]
            v = ref.silu_mul(v)
            err = err + v.abs() * 2.0 ** -20
        check(y[lo:hi], v, err, f"group {e} of {counts} {N} {K} {act}")
    return y


RAGGED = [(3,), (1, 0, 2, 0, 0, 1), (5, 16, 17, 0, 1), (0, 0, 40), (70, 3, 129, 64), (300, 0, 257), (0, 0),
          (33, 31, 1, 0, 0, 0, 0, 15, 16, 90)]


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts", RAGGED, ids=str)
def test_grouped(w4, act, gated, counts):
    if sum(counts) == 0:
        grouped_case(w4, counts, 64, 160, act, gated=gated, tail=3)
        return
    grouped_case(w4, counts, 160, 416, act, gated=gated, near=False)
    grouped_case(w4, counts, 96, 2912, act, gated=gated, tail=5, lead=2, gather=False)


MANY = [((*[(i * 7) % 4 for i in range(200)],), 64, 288), ((1,) * 16, 64, 1056), ((4, 0, 9, 1, 6, 0, 0, 3), 1056, 544),
        ((130, 60, 80), 288, 544), ((300, 250, 500), 352, 800), ((400, 500, 0, 700, 900), 544, 288),
        ((1100, 900, 0, 1300), 4128, 544)]


def grouped_sizes():
    """(counts, N, K, gated) of the tests of grouped products."""
    out = [(c, 160, 416, g) for c in RAGGED for g in (False, True) if sum(c)]
    return out + [(c, N, K, g) for c, N, K in MANY for g in (False, True)]


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("case", MANY, ids=lambda c: f"{sum(c[0])}rows_{len(c[0])}groups")
def test_grouped_of_many_groups_and_each_tile(w4, act, gated, case):
    counts, N, K = case
    grouped_case(w4, counts, N, K, act, gated=gated, tail=7)
    grouped_case(w4, counts, N, K, act, gated=gated, gather=False, tail=7, dtype="f32", rule="ceil", near=False)


@pytest.mark.parametrize("counts", [(3, 2), (20, 40), (140, 90)])
def test_grouped_rows_out_of_range_give_zeros(w4, counts):
    P = sum(counts)
    y = grouped_case(w4, counts, 64, 160, "fp4", bad=[(0, -1), (P - 1, 37), (P // 2, -2 ** 31), (1, 2 ** 31 - 1)])
    for at in (0, P - 1, P // 2, 1):
        assert bool((y[at] == 0).all())


def test_non_finite_rows_stay_in_their_row(w4):
    """A NaN or an infinity makes its own row NaN and no other."""
    for M, N, K in ((3, 64, 160), (16, 64, 544), (40, 128, 288), (130, 128, 160)):
        for act in FMTS:
            g = gen(M)
            x = torch.randn(M, K, generator=g)
            x[0, 5] = float("nan")
            x[M // 2, K - 1] = float("-inf")
            q, s = weight(g, N, K)
            w = w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda())
            y = w4.mx_linear(x.cuda(), w, act=act).cpu()
            bad = torch.zeros(M, dtype=torch.bool)
            bad[[0, M // 2]] = True
            assert bool(torch.isnan(y[bad]).all()) and bool(torch.isfinite(y[~bad]).all())


def test_a_nan_weight_scale_stays_in_its_channel(w4):
    for M, K in ((1, 160), (20, 160), (140, 672)):
        g = gen(M)
        q, s = weight(g, 64, K)
        s[21, K // 32 - 1] = 255
        w = w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda())
        y = w4.mx_linear(torch.randn(M, K, generator=g).cuda(), w).cpu()
        bad = torch.zeros(64, dtype=torch.bool)
        bad[21] = True
        assert bool(torch.isnan(y[:, bad]).all()) and bool(torch.isfinite(y[:, ~bad]).all())


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts,path", [((3, 2), 1), ((9, 0, 4) + (7,) * 6, 2), ((70, 3, 90), 3)])
def test_rows_out_of_range_give_zeros_whatever_the_weight(w4, counts, path, gated):
    """Also where the weight's scales, or row 0 of x, are NaN."""
    E, N, K, P, M = len(counts), 64, 544, sum(counts), 37
    assert w4.mx_grouped_linear_plan(M, P, E, N, K).path == path
    g = gen(P)
    q, s = weight(g, E * N, K)
    s[::5, K // 32 - 1] = 255
    w = w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda(), n_experts=E)
    x = torch.randn(M, K, generator=g)
    x[0, 7] = float("nan")
    rows = torch.randint(1, M, (P,), generator=g, dtype=torch.int32)
    bad = [0, 1, P // 2, P - 1]
    rows[bad] = torch.tensor([-1, M, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)
    offsets = torch.cumsum(torch.tensor([0] + list(counts)), 0).to(torch.int32)
    y = w4.mx_grouped_linear(x.cuda(), w, offsets.cuda(), rows=rows.cuda(), gated=gated).cpu()
    assert bool((y[bad] == 0).all())
    good = torch.ones(P, dtype=torch.bool)
    good[bad] = False
    assert bool(torch.isnan(y[good]).any(1).all()) and bool(torch.isfinite(y[good]).any(1).all())


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("per,path", [({3: 1, 127: 2, 128: 1, 700: 4, 1023: 3}, 1), ({0: 9, 511: 40, 512: 17, 1022: 3}, 2),
                                      ({0: 700, 255: 64, 256: 65, 800: 9000, 1023: 130}, 3)])
def test_grouped_of_1024_groups(w4, act, per, path):
    """The most groups: rows in the first, the last and those around the borders of the lists."""
    counts = tuple(per.get(e, 0) for e in range(1024))
    assert w4.mx_grouped_linear_plan(37, sum(counts) + 2, 1024, 64, 160, act).path == path
    grouped_case(w4, counts, 64, 160, act, tail=2)
    grouped_case(w4, counts, 64, 160, act, tail=2, gather=False, gated=True)


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("M", [1, 17, 70])
def test_most_inputs(w4, act, M):
    """K = 2^22: rows of zeros but for a few blocks, the first and the last among them, whose sums
    are as near as those of few inputs."""
    K, N = 1 << 22, 32
    g = gen(M)
    blocks = torch.randint(0, K // 32, (M, 6), generator=g)
    blocks[:, 0] = K // 32 - 1
    blocks[0, 1] = 0
    x = torch.zeros(M, K // 32, 32)
    x[torch.arange(M)[:, None], blocks] = activations(g, M, 6 * 32, True).view(M, 6, 32)
    x = x.view(M, K).to(torch.bfloat16).cuda()
    q = torch.randint(0, 16, (N, K), generator=g, dtype=torch.uint8)
    s = torch.randint(118, 123, (N, K // 32), generator=g, dtype=torch.uint8)
    w = w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda())
    y = w4.mx_linear(x, w, act=act)
    rows = w4.mx_grouped_linear(x, w, torch.tensor([0, M], dtype=torch.int32).cuda(), act=act)
    for m in range(M):
        at = (torch.unique(blocks[m])[:, None] * 32 + torch.arange(32)).reshape(-1)
        xv = ref.rounded(x[m:m + 1, at.cuda()].contiguous(), act, "floor")
        wv = ref.values(q[:, at].contiguous().cuda(), s[:, torch.unique(blocks[m])].contiguous().cuda(), "fp4")
        e, _ = ref.slack(xv, wv, act)
        for got in (y, rows):
            check(got[m:m + 1], xv @ wv.t().contiguous(), e, f"row {m}")
