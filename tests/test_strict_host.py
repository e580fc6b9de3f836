"""The strict bf16 comparison (no GPU needed; the mistakes are planted in its inputs)."""
import pytest
import torch

import expert_reference as R
import strict_reference as S

NAN, INF = float("nan"), float("inf")


def _case():
    gen = torch.Generator().manual_seed(6)
    a, w = torch.randn(9, 256, generator=gen, dtype=R.D), torch.randn(40, 256, generator=gen, dtype=R.D)
    y, bound = R.product(a, w)
    return y.bfloat16(), y, bound


def test_accepts_what_is_rounded():
    got, y, bound = _case()
    S.assert_bf16(got, y, bound * 0, "rounded")


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_refuses_one_value_that_is_not_finite(bad):
    got, y, bound = _case()
    got[2, 3] = bad
    with pytest.raises(AssertionError):
        S.assert_bf16(got, y, bound, "one")
    with pytest.raises(AssertionError):
        S.assert_bf16(torch.full_like(got, bad), y, bound, "all")


def test_refuses_a_value_that_is_a_step_off():
    got, y, bound = _case()
    got[2, 3] *= 1 + 2 ** -5
    with pytest.raises(AssertionError):
        S.assert_bf16(got, y, bound * 0, "off")


@pytest.mark.parametrize("want,right,wrong", [(NAN, NAN, 1.0), (NAN, NAN, INF), (INF, INF, -INF), (-INF, -INF, 3e38),
                                              (INF, INF, NAN)])
def test_takes_what_the_reference_has(want, right, wrong):
    got, y, bound = _case()
    y[2, 3], got[2, 3] = want, right
    S.assert_bf16(got, y, bound, "same")
    got[2, 3] = wrong
    with pytest.raises(AssertionError):
        S.assert_bf16(got, y, bound, "other")
