"""The expert-layer operators in 64 bits, and how far a correct kernel may be
from them.

Every function takes torch tensors on any device and computes in float64.
Bounds are derived, not fitted:

* a rounding is off by at most half a step, eps / 2 of its type relative to the
  value (bf16 2^-8, E4M3 2^-4; below E4M3's smallest normal half its step);
* a sum of n fp32 terms is off by at most n * 2^-24 of the sum of magnitudes;
* the 8-bit matrix instruction adds products in groups of eight adjacent
  channels and cuts each 13 binary places below the group's largest: at most
  7 * 2^-13 < 2^-10 of that one per group.
"""
import numpy as np
import torch

D = torch.float64
NONE, FP8_F32, FP8_UE8M0, MXFP8 = 0, 1, 2, 3
F8 = torch.float8_e4m3fn


def e8m0(byte):
    return torch.exp2(byte.to(D) - 127)


def group(quant):
    return 32 if quant == MXFP8 else 128


def block_scale(amax, quant):
    """The scale of blocks with largest magnitude amax (float64)."""
    a = amax.clamp_min(float(np.float32(1e-10)))
    if quant == FP8_F32:
        return a / 448
    m, e = torch.frexp(a)
    k = e - 9
    if quant == FP8_UE8M0:
        k = k + (m > 0.875).to(k.dtype)
    return torch.exp2(k.to(D))


def quantize(x, quant):
    """Rows x [.., n] -> (E4M3 bytes uint8, stored scales), by the dispatch's rules."""
    b = x.to(D).unflatten(-1, (-1, group(quant)))
    s = block_scale(b.abs().amax(-1), quant)
    if quant == FP8_F32:
        s = s.to(torch.float32).to(D)
    q = (b / s.unsqueeze(-1)).clamp(-448, 448).flatten(-2).to(torch.float32).to(F8).view(torch.uint8)
    if quant == FP8_F32:
        return q, s.to(torch.float32)
    byte = (torch.log2(s).round() + 127).to(torch.uint8)
    if quant == MXFP8:
        return q, byte
    pad = -byte.shape[-1] % 4
    return q, torch.nn.functional.pad(byte, (0, pad)).contiguous().view(torch.int32)


def scale_values(scale, quant, groups):
    """Stored scales of rows -> float64 values [.., groups]."""
    if quant == FP8_F32:
        return scale.to(D)
    return e8m0(scale.view(torch.uint8)[..., :groups])


def dequantize(q, scale, quant):
    g = group(quant)
    s = scale_values(scale, quant, q.shape[-1] // g)
    return (q.view(F8).to(D).unflatten(-1, (-1, g)) * s.unsqueeze(-1)).flatten(-2)


def weight_values(w, scale, quant):
    """Values of weights [E, n, k]."""
    if quant == NONE:
        return w.to(D)
    if quant == MXFP8:
        return dequantize(w, scale, quant)
    E, n, k = w.shape
    s = scale_values(scale, quant, k // 128).repeat_interleave(128, 1)[:, :n]
    return (w.view(F8).to(D).unflatten(-1, (-1, 128)) * s.unsqueeze(-1)).flatten(-2)


def make_weights(gen, E, n, k, quant, device="cpu"):
    """Random weights [E, n, k] in a weight format: (w, w_scale)."""
    v = torch.randn(E, n, k, generator=gen, device=device)
    if quant == NONE:
        return (v / k ** 0.5).bfloat16(), None
    w = (v * 90).clamp(-448, 448).to(F8).view(torch.uint8)
    at = 127 - round(np.log2(90 * k ** 0.5))
    if quant == FP8_F32:
        return w, (0.5 + torch.rand(E, -(-n // 128), k // 128, generator=gen, device=device)) / (90 * k ** 0.5)
    if quant == MXFP8:
        return w, torch.randint(at - 2, at + 2, (E, n, k // 32), generator=gen, device=device).to(torch.uint8)
    nb = k // 128
    s = torch.zeros(E, -(-n // 128), -(-nb // 4) * 4, dtype=torch.uint8, device=device)
    s[..., :nb] = torch.randint(at - 2, at + 2, (E, s.shape[1], nb), generator=gen, device=device).to(torch.uint8)
    return w, s.view(torch.int32)


def silu(v):
    return v * torch.sigmoid(v)


def product(a, w, eight_bit=True):
    """a [m, k] @ w [n, k].T in float64, and a bound on a kernel's fp32 result:
    8-bit products (the groups of eight) and the fp32 sums of k terms."""
    y = a @ w.T
    m, k = a.shape
    mag = a.abs() @ w.abs().T
    bound = (k + 8) * 2.0 ** -24 * mag
    if eight_bit:
        step = max(1, (1 << 24) // max(1, w.numel()))
        wg = w.abs().unflatten(1, (-1, 8))
        for i in range(0, m, step):
            ag = a[i:i + step].abs().unflatten(1, (-1, 8))
            bound[i:i + step] += 2.0 ** -10 * (ag[:, None] * wg[None]).amax(-1).sum(-1)
    return y, bound


def assert_bf16(got, want, bound, what):
    """got = bf16(want with an error of at most `bound`)."""
    lim = (want.abs() + bound) * 2.0 ** -8 + bound
    err = (got.to(D) - want).abs()
    bad = err > lim
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                                 f"{float((err / lim.clamp_min(1e-300)).max()):.2f} times the bound")


def assert_rows(q, scale, want, bound, quant, what):
    """(q, scale) = quantization of `want` known to within `bound`."""
    g = group(quant)
    groups = want.shape[-1] // g
    s = scale_values(scale, quant, groups)
    amax, d = want.abs().unflatten(-1, (-1, g)).amax(-1), bound.unflatten(-1, (-1, g)).amax(-1)
    lo, hi = block_scale((amax - d).clamp_min(0), quant), block_scale(amax + d, quant)
    tol = 2.0 ** -22 if quant == FP8_F32 else 0.0  # a division and a stored fp32 value
    ok = (s >= lo * (1 - tol)) & (s <= hi * (1 + tol))
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} of {ok.numel()} scales off"
    sx = s.repeat_interleave(g, -1)
    top = 448 * sx
    got = q.view(F8).to(D) * sx
    inside = want.clamp(min=-top, max=top)
    lim = bound + (inside.abs() + bound) * 2.0 ** -4 + sx * 2.0 ** -10
    err = (got - inside).abs()
    assert bool((err <= lim).all()), (f"{what}: {int((err > lim).sum())} of {err.numel()} values off, worst "
                                      f"{float((err / lim).max()):.2f} times the bound")
