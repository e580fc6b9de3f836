"""The bf16 expert layer and its gradients in 64 bits, and how far a correct
kernel may be from them.

Bounds are derived, not fitted (see expert_reference for the roundings):

* a sum of n fp32 terms is off by at most n * 2^-23 of the sum of magnitudes: one
  rounding per term, or a cut of a whole step where the matrix instruction drops
  low bits instead of rounding;
* exp, the quotient and the products of an activation cost at most 2^-21 of the
  larger of its argument and value: exp's argument z is off by 2^-22 |z|, which
  s (1 - s) |z| < 0.23 damps; its input's error passes with a slope of at most 1.13;
* a slope is off by at most 2^-18: 1 - s is off by 2^-24, times c z'(c) < 35 where
  s still differs from 1 in 32 bits (c < 5), and the errors of s as above.
"""
import math

import torch

import expert_reference as R

D = torch.float64
NONE, SILU, GELU, RELU = 0, 1, 2, 3


def act(v, kind):
    """An activation and its slope."""
    if kind == SILU:
        s = torch.sigmoid(v)
        return v * s, s * (1 + v * (1 - s))
    if kind == GELU:
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (v + 0.044715 * v ** 3))
        return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)
    if kind == RELU:
        return torch.where(v > 0, v, torch.zeros_like(v)), (v > 0).to(D)
    return v, torch.ones_like(v)


def product(a, w):
    """a [m, k] @ w [n, k].T and the bound of its fp32 sum."""
    k = a.shape[1]
    return a @ w.T, (k + 8) * 2.0 ** -23 * (a.abs() @ w.abs().T)


def gated(p, bound, kind):
    """act(gate) * up of products known to within `bound`."""
    (g, u), (bg, bu) = p.chunk(2, -1), bound.chunk(2, -1)
    f, _ = act(g, kind)
    bf = act_bound(g, f, bg, kind)
    return f * u, bf * (u.abs() + bu) + f.abs() * bu + (f * u).abs() * 2.0 ** -23


def act_bound(v, f, bound, kind):
    if kind in (NONE, RELU):
        return bound
    return 1.13 * bound + (v.abs() + f.abs()) * 2.0 ** -21


def act_grads(dy, saved, kind, is_gated):
    """(dsaved, y) with their bounds before rounding; saved is exact."""
    if not is_gated:
        f, s = act(saved, kind)
        slope = 0.0 if kind in (NONE, RELU) else 2.0 ** -18
        ds = dy * s
        return (ds, dy.abs() * slope + ds.abs() * 2.0 ** -22), (f, act_bound(saved, f, torch.zeros_like(f), kind))
    g, u = saved.chunk(2, -1)
    f, s = act(g, kind)
    slope = 0.0 if kind in (NONE, RELU) else 2.0 ** -18
    bf = act_bound(g, f, torch.zeros_like(f), kind)
    dg, du, y = dy * u * s, dy * f, f * u
    bg = (dy * u).abs() * slope + dg.abs() * 2.0 ** -21
    bu = dy.abs() * bf + du.abs() * 2.0 ** -23
    by = u.abs() * bf + y.abs() * 2.0 ** -23
    return (torch.cat([dg, du], -1), torch.cat([bg, bu], -1)), (y, by)


def assert_near(got, want, bound, what):
    """got (fp32) within `bound` of want, and half a step of fp32."""
    lim = bound + want.abs() * 2.0 ** -23
    err = (got.to(D) - want).abs()
    bad = ~(err <= lim)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                                 f"{float((err / lim.clamp_min(1e-300)).max()):.2f} times the bound")


assert_bf16, assert_rows, dequantize, quantize = R.assert_bf16, R.assert_rows, R.dequantize, R.quantize
