"""CPU: the comparison of mx_strict.py accepts correctly rounded values and refuses
every other, NaN and infinities among them."""
import pytest
import torch

import mx_strict


def parts():
    want = torch.tensor([[1.0, -2.5, 0.0], [3e-39, 7e38, -7e38]], dtype=torch.float64)
    return want.float().to(torch.bfloat16), want, torch.zeros_like(want)


def test_rounded_values_pass():
    mx_strict.check(*parts())
    y, want, err = parts()
    want[0, 0] = y[0, 0] = float("nan")
    mx_strict.check(y, want, err)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), 1.02])
@pytest.mark.parametrize("at", [(0, 0), (0, 2), (1, 0)])
def test_other_values_do_not(value, at):
    y, want, err = parts()
    y[at] = value
    with pytest.raises(AssertionError):
        mx_strict.check(y, want, err)


@pytest.mark.parametrize("value", [float("nan"), float("-inf"), 3.3e38])
def test_a_sum_past_the_largest_value_is_its_infinity(value):
    y, want, err = parts()
    y[1, 1] = value
    with pytest.raises(AssertionError):
        mx_strict.check(y, want, err)


def test_an_output_of_nans_is_refused():
    y, want, err = parts()
    with pytest.raises(AssertionError):
        mx_strict.check(torch.full_like(y, float("nan")), want, err + 1e30)


def test_a_nan_is_not_a_number():
    y, want, err = parts()
    want[0, 0] = float("nan")
    with pytest.raises(AssertionError):
        mx_strict.check(y, want, err)
