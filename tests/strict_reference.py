"""The bf16 comparison of expert_reference for results that have to be numbers.

There a result is refused whose error is larger than its limit.  The error of a
NaN is NaN, which is larger than nothing, so a NaN passes.  Here a result is
accepted whose error is within its limit, and one that is not finite only
where the reference is the same."""
import torch

import expert_reference as R


def assert_bf16(got, want, bound, what):
    """got = bf16(want with an error of at most `bound`); NaN and infinities only where want has them."""
    lim = (want.abs() + bound) * 2.0 ** -8 + bound
    err = (got.to(R.D) - want).abs()
    ok = torch.where(want.isfinite(), err <= lim, (got.to(R.D) == want) | (got.isnan() & want.isnan()))
    assert bool(ok.all()), (f"{what}: {int((~ok).sum())} of {ok.numel()} off, {int((got.isnan() & ~ok).sum())} of them NaN, "
                            f"worst {float((err / lim.clamp_min(1e-300)).nan_to_num(0.0).max()):.2f} times the bound")
