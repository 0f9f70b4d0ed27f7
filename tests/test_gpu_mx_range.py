"""GPU: microscaled products near the ends of the exponent range: subnormal sums,
scales far from one whose products are ordinary, sums past float32's largest value.

Definitions are those of test_gpu_mx.py, the comparison that of mx_strict.py.  A
float32 sum of subnormal products is off by at most 2^-149 an addition more than
the slack counts; bfloat16's half step down there is 2^-134, and the comparison
allows 2^-133, so that 2^15 additions fit.
"""
import pytest

torch = pytest.importorskip("torch")

import mx_reference as ref  # noqa: E402
import mx_strict  # noqa: E402
from test_gpu_mx import FMTS, activations, gen, w4  # noqa: E402,F401

pytestmark = pytest.mark.gpu

# binades by which rows and weights are moved from one
ENDS = [(-64, -66), (-66, -68), (-100, -27), (-122, 120), (-120, 0), (120, -120), (124, -110), (6, -122)]
PAST = [(62, 60), (100, 40), (120, 120)]
# (rows, channels, inputs): raw rows, streams, every tile, slices
SIZES = [(1, 64, 672), (16, 64, 1056), (16, 4112, 2080), (40, 256, 1056), (20, 8208, 1056), (65, 4112, 672),
         (200, 8208, 288), (300, 18960, 416), (1030, 12816, 288), (33, 256, 9248), (513, 528, 16416)]
# (rows of each group, channels, inputs): raw rows, stream, every tile
GROUPS = [((1, 0, 2, 1), 64, 1056), ((4, 0, 9, 1, 6, 0, 0, 3), 96, 2080), ((70, 3, 90), 288, 544),
          ((300, 250, 500), 352, 800), ((1100, 900), 544, 288)]


def weight(g, N, K, ew, positive):
    q = torch.randint(0, 8 if positive else 16, (N, K), generator=g, dtype=torch.uint8)
    s = torch.randint(127 + ew - 1, 127 + ew + 2, (N, K // 32), generator=g, dtype=torch.uint8)
    return q, s


def rows_of(g, M, K, ex, positive):
    x = activations(g, M, K, True)
    return torch.ldexp(x.abs() if positive else x, torch.tensor(ex)).to(torch.bfloat16).cuda()


def linear(w4, size, act, ex, ew, positive=False):  # noqa: F811
    M, N, K = size
    g = gen(M + N + K)
    x, (q, s) = rows_of(g, M, K, ex, positive), weight(g, N, K, ew, positive)
    y = w4.mx_linear(x, w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda()), act=act)
    xv, wv = ref.rounded(x, act, "floor"), ref.values(q.cuda(), s.cuda(), "fp4")
    want = xv @ wv.t().contiguous()
    mx_strict.check(y, want, ref.slack(xv, wv, act)[0], f"{size} {act} 2^{ex} 2^{ew}")
    return want


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_linear_near_the_ends(w4, act, size):  # noqa: F811
    for ex, ew in ENDS:
        linear(w4, size, act, ex, ew)


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sums_past_the_largest_value(w4, act, size):  # noqa: F811
    """Terms of one sign: every sum is an infinity, none is NaN."""
    for ex, ew in PAST:
        assert float(linear(w4, size, act, ex, ew, positive=True).min()) > 2.0 ** 128


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("case", GROUPS, ids=lambda c: f"{sum(c[0])}rows")
def test_groups_near_the_ends(w4, act, gated, case):  # noqa: F811
    """Gated: outputs that are subnormal, gates so far below zero that nothing is left of them, and
    so far above that the output is their product with the value."""
    counts, N, K = case
    E, P = len(counts), sum(counts)
    offsets = torch.cumsum(torch.tensor([0] + list(counts)), 0).to(torch.int32)
    for ex, ew in [(-30, -34), (-40, -24), (100, -48), (-70, 124), (28, 24)] if gated else ENDS:
        g = gen(P + N + K)
        x, (q, s) = rows_of(g, P, K, ex, False), weight(g, E * N, K, ew, False)
        w = w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda(), n_experts=E)
        y = w4.mx_grouped_linear(x, w, offsets.cuda(), gated=gated, act=act)
        xv, wv = ref.rounded(x, act, "floor"), ref.values(q.cuda(), s.cuda(), "fp4")
        for e in range(E):
            run = slice(int(offsets[e]), int(offsets[e + 1]))
            if run.start == run.stop:
                continue
            we = wv[e * N:(e + 1) * N]
            v, (err, _) = xv[run] @ we.t().contiguous(), ref.slack(xv[run], we, act)
            if gated:
                h = N // 2
                gate, val = v[:, :h], v[:, h:]
                err = 1.1 * err[:, :h] * val.abs() + gate.abs() * err[:, h:] + 1.1 * err[:, :h] * err[:, h:]
                v = ref.silu_mul(v)
                err = err + v.abs() * 2.0 ** -20
            mx_strict.check(y[run], v, err, f"group {e} 2^{ex} 2^{ew}")


@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("counts", [(2, 0, 1), (9, 4, 0, 3), (70, 3, 90)])
def test_a_gate_past_the_smallest_value_is_nan(w4, act, counts):  # noqa: F811
    """As the header states: the sum is minus infinity, and its sigmoid's product NaN; the gates
    beside it are their own."""
    E, N, K = len(counts), 64, 544
    g = gen(sum(counts))
    q, s = weight(g, E * N, K, 60, True)
    q[::4] |= 8  # of every four gates (and values) one is negative
    offsets = torch.cumsum(torch.tensor([0] + list(counts)), 0).to(torch.int32)
    w = w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda(), n_experts=E)
    y = w4.mx_grouped_linear(rows_of(g, sum(counts), K, 62, True), w, offsets.cuda(), gated=True, act=act).cpu()
    low = torch.arange(N // 2) % 4 == 0
    assert bool(torch.isnan(y[:, low]).all()) and bool((y[:, ~low] == float("inf")).all())
