"""Comparison of bfloat16 outputs with 64-bit sums that nothing but equal special
values passes: a NaN, or an infinity where the sum is finite, is an error."""
import torch


def check(y, want, err, name=""):
    """bf16 y against 64-bit sums `want` that float32 may miss by err, rounded once.

    Sums that round to a bfloat16 infinity have to be that infinity; those of
    NaN have to be NaN."""
    y, want, err = y.double().cpu(), want.cpu(), err.cpu()
    bound = want.abs() * 2.0 ** -8 + err * (1 + 2.0 ** -8) + 2.0 ** -133
    past = want.to(torch.float32).to(torch.bfloat16).double()
    good = (y - want).abs() <= bound
    good &= ~torch.isinf(y)
    good |= torch.isinf(past) & (y == past)
    good |= torch.isnan(want) & torch.isnan(y)
    bad = ~good
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()}, first {torch.nonzero(bad)[0].tolist()}, " \
                          f"{y[bad][0]} against {want[bad][0]} (bound {bound[bad][0]})"
