"""GPU: ragged products whose offsets lie outside the rows or fall.  Every offset is
bounded to the rows and a run that falls is empty; the bounded runs have the
products of their own groups, rows of no run stay as they were.

Definitions are those of test_gpu_mx.py, the comparison that of mx_strict.py.
"""
import pytest

torch = pytest.importorskip("torch")

import mx_reference as ref  # noqa: E402
import mx_strict  # noqa: E402
from test_gpu_mx import FMTS, activations, gen, w4, weight  # noqa: E402,F401

pytestmark = pytest.mark.gpu

BIG = 2 ** 31 - 1
SIZES = [(3, 12), (40, 60), (3, 100), (3, 400), (2, 1600), (12, 60), (5, 2000)]


def patterns(E, P):
    first = P // 2
    rest = [[BIG] * E, [-5] * E, [P] * E, [0, BIG] * E, [first, -BIG - 1, BIG] * E, [first + 3, BIG] + [BIG] * E]
    return [([0, first] + r)[:E + 1] for r in rest] + [([-BIG - 1, first, BIG] + [BIG] * E)[:E + 1]]


def runs(offsets, P):
    bounded = [min(max(o, 0), P) for o in offsets]
    return [(lo, max(lo, hi)) for lo, hi in zip(bounded, bounded[1:])]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", FMTS)
@pytest.mark.parametrize("E,P", SIZES)
def test_bounded_runs_have_their_own_products(w4, act, E, P, gated):  # noqa: F811
    K, N = 160, 64
    g = gen(E + P)
    x = activations(g, P, K, True).to(torch.bfloat16).cuda()
    q, s = weight(g, E * N, K)
    w = w4.mx_pack_weights(ref.pack4(q).cuda(), s.cuda(), n_experts=E)
    xv, wv = ref.rounded(x, act, "floor"), ref.values(q.cuda(), s.cuda(), "fp4")
    plan = w4.mx_grouped_linear_plan(P, P, E, N, K, act)
    width = N // 2 if gated else N
    for offsets in patterns(E, P):
        buf = torch.full((P + 64, width), 7.5, dtype=torch.bfloat16, device="cuda")
        y = buf[32:32 + P]
        w4.mx_grouped_linear(x, w, torch.tensor(offsets, dtype=torch.int32).cuda(), gated=gated, act=act, out=y)
        assert bool((buf[:32] == 7.5).all()) and bool((buf[32 + P:] == 7.5).all())
        own = runs(offsets, P)
        named = torch.zeros(P, dtype=torch.int32)
        for lo, hi in own:
            named[lo:hi] += 1
        assert bool((y.cpu()[named == 0] == 7.5).all()), offsets
        # (more tiles than sound offsets can have are not all worked on)
        tiles = sum(-(-(hi - lo) // plan.tile_rows) for lo, hi in own)
        if tiles > -(-P // plan.tile_rows) + min(E, P):
            assert any(b < a for a, b in zip(offsets, offsets[1:]))
            continue
        for e, (lo, hi) in enumerate(own):
            alone = torch.arange(lo, hi)[named[lo:hi] == 1].cuda()
            if not len(alone):
                continue
            we = wv[e * N:(e + 1) * N]
            v, (err, _) = xv[alone] @ we.t().contiguous(), ref.slack(xv[alone], we, act)
            if gated:
                gate, val, h = v[:, :width], v[:, width:], width
                err = 1.1 * err[:, :h] * val.abs() + gate.abs() * err[:, h:] + 1.1 * err[:, :h] * err[:, h:]
                v = ref.silu_mul(v)
                err = err + v.abs() * 2.0 ** -20
            mx_strict.check(y[alone], v, err, f"group {e} of {offsets[:6]}")


def test_patterns_name_what_they_mean():
    """Of the patterns: one whose second run is bounded, ones that fall, rows of no run."""
    for E, P in SIZES:
        found = [(o, runs(o, P)) for o in patterns(E, P)]
        assert any(BIG in o and r[1] == (P // 2, P) for o, r in found)
        assert any(any(b < a for a, b in zip(o, o[1:])) for o, _ in found)
        assert any(sum(hi - lo for lo, hi in r) < P for _, r in found)
