"""The expert-layer operators where they can go wrong: values that are not
finite, channels that cancel, long sums, kernel variants that need large calls.

Compared with 64-bit references (tests/expert_reference.py) or with the bytes of
a call that must agree.  Every comparison fails on a NaN it does not ask for.
Every test prints the case it runs before touching the GPU.
"""
import pytest
import torch

import combine_topk_idx_amd as M
import expert_reference as R
from test_gpu_experts import _cfg, _filled, _gen, _gpu, _say, _scales  # noqa: F401 (_gpu: a fixture)

pytestmark = pytest.mark.gpu
D = R.D
FORMATS = [M.QUANT_FP8_F32, M.QUANT_FP8_UE8M0, M.QUANT_MXFP8]
INF, NAN = float("inf"), float("nan")


def _is_nan(q):
    """E4M3 NaN, of either sign."""
    return (q & 0x7F) == 0x7F


def _bytes_equal(a, b, what):
    assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), what


# ---- values that are not finite ----------------------------------------------------------


def _norm(x, w, quant, residual=None):
    T, H = x.shape
    out, q, s = _filled((T, H), torch.bfloat16), _filled((T, H), torch.uint8), _scales(T, H, quant)
    res_out = None if residual is None else _filled((T, H), torch.bfloat16)
    M.moe_rmsnorm(_cfg(T, H, quant=quant), T, x, residual, w, 1e-6, res_out, out, q, s)
    torch.cuda.synchronize()
    return out, q, s


@pytest.mark.parametrize("quant", FORMATS)
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_rmsnorm_of_a_token_that_is_not_finite(bad, quant):
    """NaN in a row: all of it.  An infinity: the mean of squares is infinite, so that channel is NaN and
    the others are 0.  The other rows are as without it."""
    _say(f"rmsnorm, one channel of one token {bad}, quant={quant}")
    g = _gen(3)
    x = torch.randn(5, 640, generator=g, device="cuda").bfloat16()
    w = torch.randn(640, generator=g, device="cuda").bfloat16()
    clean = _norm(x, w, quant)
    x2 = x.clone()
    x2[2, 300] = bad
    got = _norm(x2, w, quant)
    for a, b in zip(got, clean):
        _bytes_equal(a[[0, 1, 3, 4]], b[[0, 1, 3, 4]], "another token")
    out, q = got[0][2], got[1][2]
    at = torch.zeros(640, dtype=torch.bool, device="cuda")
    at[300] = True
    if bad != bad:
        at[:] = True
    assert torch.equal(out.isnan(), at) and torch.equal(_is_nan(q), at)
    assert not bool((q[~at] & 0x7F).any())


@pytest.mark.parametrize("quant", FORMATS)
def test_rmsnorm_with_a_weight_that_is_not_finite(quant):
    """A NaN weight makes its channel NaN; scale and bytes of the others are those of a channel that is 0."""
    _say(f"rmsnorm, one weight NaN, quant={quant}")
    g = _gen(4)
    x = torch.randn(7, 512, generator=g, device="cuda").bfloat16()
    w = torch.randn(512, generator=g, device="cuda").bfloat16()
    w[130] = 0.0
    zero = _norm(x, w, quant)
    w[130] = NAN
    out, q, s = _norm(x, w, quant)
    _bytes_equal(s, zero[2], "scales")
    rest = torch.arange(512, device="cuda") != 130
    _bytes_equal(q[:, rest], zero[1][:, rest], "other channels")
    assert bool(_is_nan(q[:, 130]).all()) and bool(out[:, 130].isnan().all()) and not bool(out[:, rest].isnan().any())


@pytest.mark.parametrize("quant", FORMATS)
def test_rmsnorm_past_the_range_of_fp32(quant):
    """A channel whose normed value is infinite: NaN beside an infinite fp32 scale, else the largest E4M3
    value, with its sign, beside 2^120; the other blocks are as they were."""
    _say(f"rmsnorm, one channel past fp32's range, quant={quant}")
    x = torch.ones(2, 256, device="cuda").bfloat16()
    x[:, 5] = 64.0            # 64 / sqrt((64^2 + 255) / 256) = 15.5 times the weight
    x[1] *= -1.0
    w = torch.ones(256, device="cuda").bfloat16()
    clean = _norm(x, w, quant)
    w[5] = 3.0e38
    out, q, s = _norm(x, w, quant)
    block = 32 if quant == M.QUANT_MXFP8 else 128
    _bytes_equal(q[:, block:], clean[1][:, block:], "other blocks")
    assert out[0, 5] == INF and out[1, 5] == -INF
    if quant == M.QUANT_FP8_F32:
        assert bool((s[:, 0] == INF).all()) and bool(_is_nan(q[:, 5]).all())
    else:
        assert s.view(torch.uint8)[:, 0].tolist() == [247, 247]  # 2^(247 - 127)
        assert q[:, 5].tolist() == [0x7E, 0xFE]
    rest = torch.arange(block, device="cuda") != 5
    assert not bool((q[:, :block][:, rest] & 0x7F).any())


@pytest.mark.parametrize("quant", FORMATS)
@pytest.mark.parametrize("T", [3, 150])
def test_products_of_a_row_with_nan(T, quant):
    """One NaN among a row's inputs: every channel of its product, of its SwiGLU rows and of their product is
    NaN, the other rows' bytes are as without it."""
    _say(f"products, T={T}, one input NaN, quant={quant}")
    k, inter = 384, 256
    g = _gen(T)
    a, s = R.quantize(torch.randn(T, k, generator=g, device="cuda"), quant)
    w13, s13 = R.make_weights(g, 1, 2 * inter, k, quant, "cuda")
    w2, s2 = R.make_weights(g, 1, k, inter, quant, "cuda")
    cfg = _cfg(T, k, quant=quant)

    def run(a):
        y, h, hs = _filled((T, 2 * inter), torch.bfloat16), _filled((T, inter), torch.uint8), _scales(T, inter, quant)
        z = _filled((T, k), torch.bfloat16)
        M.moe_expert_gemm(cfg, T, 2 * inter, k, a, s, w13, s13, None, y)
        M.moe_expert_gemm_swiglu(cfg, T, inter, a, s, w13, s13, None, h, hs)
        M.moe_expert_gemm(cfg, T, k, inter, h, hs, w2, s2, None, z)
        torch.cuda.synchronize()
        return y, h, hs, z

    clean = run(a)
    bad = a.clone()
    bad[1, 200] = 0x7F
    got = run(bad)
    rest = torch.arange(T, device="cuda") != 1
    for i, (u, v) in enumerate(zip(got, clean)):
        _bytes_equal(u[rest], v[rest], f"another row of output {i}")
    assert bool(got[0][1].isnan().all()) and bool(_is_nan(got[1][1]).all()) and bool(got[3][1].isnan().all())


# ---- sums -----------------------------------------------------------------------------------


def _cancelling(T, blocks, n, g):
    """E4M3 rows [T, 128 blocks] and weights [n, 128 blocks] of whole numbers, whose products and partial sums
    are whole numbers below 2^24 (exact in fp32 in any order).  Row r has, in block r % blocks, two adjacent
    channels whose products with every weight are 448^2 and -448^2; the rest are products of -1, 0 and 1."""
    k = 128 * blocks
    a = torch.randint(-1, 2, (T, k), generator=g, device="cuda").float()
    w = torch.randint(-1, 2, (n, k), generator=g, device="cuda").float()
    w *= (torch.rand(n, k, generator=g, device="cuda") < 0.2)
    loud = 128 * torch.arange(blocks, device="cuda") + 40
    a[:, loud] = 0.0
    a[:, loud + 1] = 0.0
    w[:, loud] = 448.0
    w[:, loud + 1] = -448.0
    r = torch.arange(T, device="cuda")
    a[r, loud[r % blocks]] = 448.0
    a[r, loud[r % blocks] + 1] = 448.0
    return a, w


@pytest.mark.parametrize("T", [5, 33, 100, 300])
def test_swiglu_rows_with_fp32_scales_come_of_fp32_sums(T):
    """Loud channels that cancel, in each of seven blocks: what is left of the sum is what is beside them."""
    _say(f"expert_gemm_swiglu of cancelling channels, T={T}")
    quant, inter, blocks = M.QUANT_FP8_F32, 256, 7
    g = _gen(T)
    a, w = _cancelling(T, blocks, 2 * inter, g)
    y = a.double() @ w.double().T
    assert float(y.abs().max()) < 60.0 and float(y.abs().mean()) > 3.0
    to8 = lambda v: v.to(R.F8).view(torch.uint8)  # noqa: E731
    s = torch.ones(T, blocks, device="cuda")
    ws = torch.ones(1, 2 * inter // 128, blocks, device="cuda")
    h, hs = _filled((T, inter), torch.uint8), _scales(T, inter, quant)
    M.moe_expert_gemm_swiglu(_cfg(T, 128 * blocks, quant=quant), T, inter, to8(a), s, to8(w)[None], ws, None, h, hs)
    torch.cuda.synchronize()
    gate, up = y[:, :inter], y[:, inter:]
    want = R.silu(gate) * up
    # exact sums; the function itself in fp32 (an exponential of argument g: |g| ulps)
    R.assert_rows(h, hs, want, want.abs() * (8 + gate.abs()) * 2.0 ** -24, quant, "h")


@pytest.mark.parametrize("quant", FORMATS)
def test_a_swiglu_row_does_not_depend_on_the_rows_beside_it(quant):
    """The same row in calls of every size: the same bytes."""
    _say(f"expert_gemm_swiglu of 1 .. 300 rows, quant={quant}")
    k, inter, T = 1152, 256, 300
    g = _gen(9)
    a, s = R.quantize(torch.randn(T, k, generator=g, device="cuda"), quant)
    w, ws = R.make_weights(g, 1, 2 * inter, k, quant, "cuda")
    full = None
    for t in (300, 129, 128, 127, 97, 96, 65, 64, 33, 32, 17, 1):
        h, hs = _filled((t, inter), torch.uint8), _scales(t, inter, quant)
        M.moe_expert_gemm_swiglu(_cfg(t, k, quant=quant), t, inter, a[:t], s[:t], w, ws, None, h, hs)
        torch.cuda.synchronize()
        if full is None:
            full = h, hs
        _bytes_equal(h, full[0][:t], f"{t} rows")
        _bytes_equal(hs, full[1][:t], f"scales of {t} rows")


@pytest.mark.parametrize("quant", FORMATS)
@pytest.mark.parametrize("T,n", [(5, 264), (130, 520), (2400, 8200)])
def test_products_of_cancelling_channels_stay_within_the_stated_bound(T, n, quant):
    """16-row strips, 128-row and 256-row tiles: each group of eight adjacent channels is off by at most
    7 * 2^-13 of its largest product, and by nothing where that one is small."""
    _say(f"expert_gemm of cancelling channels, T={T}, n={n}, quant={quant}")
    blocks = 7
    g = _gen(T + n)
    a, w = _cancelling(T, blocks, n, g)
    a[::2] = torch.where(a[::2].abs() > 1, torch.zeros_like(a[::2]), a[::2])  # rows without a loud channel
    k = 128 * blocks
    to8 = lambda v: v.to(R.F8).view(torch.uint8)  # noqa: E731
    words = {M.QUANT_FP8_F32: lambda r: torch.ones(r, blocks, device="cuda"),
             M.QUANT_FP8_UE8M0: lambda r: torch.full((r, 8), 127, dtype=torch.uint8, device="cuda").view(torch.int32),
             M.QUANT_MXFP8: lambda r: torch.full((r, k // 32), 127, dtype=torch.uint8, device="cuda")}[quant]
    y = _filled((T, n), torch.bfloat16)
    M.moe_expert_gemm(_cfg(T, k, quant=quant), T, n, k, to8(a), words(T),
                      to8(w)[None], words(n if quant == M.QUANT_MXFP8 else -(-n // 128))[None], None, y)
    torch.cuda.synchronize()
    want = a.double() @ w.double().T
    err = (y.double() - want).abs()
    half_step = want.abs() * 2.0 ** -8
    assert bool((err[::2] <= half_step[::2]).all()), "rows without loud channels"
    # every weight is loud (448) at the one loud channel of the other rows
    assert bool((err <= half_step + (1 + 2.0 ** -8) * 7 * 2.0 ** -13 * 448.0 ** 2).all())


@pytest.mark.parametrize("H", [2048, 8192])
def test_rmsnorm_keeps_small_squares_beside_large_ones(H):
    """Every thread's first channel is 4096 and its 31 others 1: added one by one to 2^24 the ones are lost.

    In fp32 the sum of a thread's four vectors may lose 3 of the 31 (a chain of four terms starts at 2^24); the
    sums of threads are equal, so that adding them is exact.  Relative to the scale, in units of 2^-24: 1.5 for
    those 3, half of one each for + eps and / H (under the root), one each for the root, the reciprocal, the
    product with it, the division by 448 and the comparison: at most 7.5.  All 31 lost are 15.5."""
    _say(f"rmsnorm, H={H}, squares of 2^24 and 1")
    x = torch.ones(3, H, device="cuda")
    x[:, 0:H // 4:8] = 4096.0
    w = torch.ones(H, device="cuda").bfloat16()
    _, _, s = _norm(x.bfloat16(), w, M.QUANT_FP8_F32)
    y = x.double() / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-6)
    want = y.unflatten(-1, (-1, 128)).amax(-1) / 448
    assert float(((s.double() - want).abs() / want).max()) <= 8.5 * 2.0 ** -24


# ---- large calls ------------------------------------------------------------------------------


def test_rmsnorm_of_more_rows_than_a_grid_holds():
    """64 threads a row: 2^26 rows are 2^32 threads, more than one launch takes."""
    T, H = (1 << 26) + 5, 8
    _say(f"rmsnorm, T={T}, H={H}")
    base = torch.randn(4099, H, generator=_gen(1), device="cuda").bfloat16()
    w = torch.randn(H, generator=_gen(2), device="cuda").bfloat16()
    cfg = _cfg(4099, H, quant=M.QUANT_NONE)
    want = _filled((4099, H), torch.bfloat16)
    M.moe_rmsnorm(cfg, 4099, base, None, w, 1e-6, None, want)
    x, out, n = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), _filled((T + 1, H), torch.bfloat16), T // 4099
    x[:n * 4099].view(n, 4099, H).copy_(base)
    x[n * 4099:].copy_(base[:T - n * 4099])
    M.moe_rmsnorm(_cfg(T, H, quant=M.QUANT_NONE), T, x, None, w, 1e-6, None, out)
    torch.cuda.synchronize()
    for i in range(0, T, 4099):
        m = min(4099, T - i)
        assert torch.equal(out[i:i + m].view(torch.int16), want[:m].view(torch.int16)), i
    assert bool((out[T:].view(torch.uint8) == 0xA5).all())


# ---- refusals -----------------------------------------------------------------------------------


def test_an_unknown_format_is_the_librarys_argument_error():
    _say("expert-layer operators with cfg.quant = 7")
    cfg = _cfg(4, 256, 2, 1, quant=7)
    b16, b8 = torch.zeros(4, 256, device="cuda").bfloat16(), torch.zeros(4, 256, dtype=torch.uint8, device="cuda")
    w = torch.zeros(2, 512, 256, dtype=torch.uint8, device="cuda")
    s = torch.zeros(2048, device="cuda")
    idx, tw = torch.zeros(4, 1, dtype=torch.int32, device="cuda"), torch.zeros(4, 1, device="cuda")
    handle = M.Handle(_cfg(4, 256, 2, 1, quant=M.QUANT_NONE))
    for call in (lambda: M.moe_rmsnorm(cfg, 4, b16, None, b16, 1e-6, None, b16, b8, s),
                 lambda: M.moe_expert_gemm(cfg, 4, 256, 256, b8, s, w, s, handle, b16),
                 lambda: M.moe_expert_gemm_swiglu(cfg, 4, 256, b8, s, w, s, handle, b8, s),
                 lambda: M.moe_layer_fused(cfg, 4, 256, idx, tw, b16, w, s, w, s, w, b16)):
        with pytest.raises(M.MoeError) as e:
            call()
        assert e.value.code == M.MOE_ERR_INVALID_ARG


def test_no_token_needs_no_buffer():
    _say("expert-layer operators without tokens or buffers")
    cfg = _cfg(4, 256, quant=M.QUANT_FP8_F32)
    w = torch.ones(256, device="cuda").bfloat16()
    M.moe_rmsnorm(cfg, 0, None, None, w, 1e-6, None, None)
    M.moe_expert_gemm(cfg, 0, 256, 256, None, None, None, None, None, None)
    M.moe_expert_gemm_swiglu(cfg, 0, 256, None, None, None, None, None, None, None)
    M.moe_layer_fused(cfg, 0, 256, None, None, None, None, None, None, None, None, None)
    with pytest.raises(M.MoeError) as e:
        x = torch.zeros(1, 256, device="cuda").bfloat16()
        w8 = torch.zeros(1, 512, 256, dtype=torch.uint8, device="cuda")
        one = torch.zeros(1, dtype=torch.int32, device="cuda")
        M.moe_layer_fused(cfg, 1, 256, one, one, x, w8, torch.zeros(8, device="cuda"), w8,
                          torch.zeros(8, device="cuda"), None, x)
    assert e.value.code == M.MOE_ERR_INVALID_ARG


# ---- exponent bytes at their ends ------------------------------------------------------------------


@pytest.mark.parametrize("quant", [M.QUANT_FP8_UE8M0, M.QUANT_MXFP8])
@pytest.mark.parametrize("byte", [3, 4, 64, 190, 246, 255])
def test_layer_weights_at_the_ends_of_their_exponents(byte, quant):
    """Every finite E4M3 value times 2^(byte - 127) as a weight, beside an h of 2^-8 or 2^8: the exact product."""
    _say(f"layer_fused, exponent byte {byte}, quant={quant}")
    H = inter = 256
    g0 = 16.0                                    # silu(16) = 16 (1 - 1.1e-7): bf16(16 u) exactly 16 u
    u = 2.0 ** -4 * (2.0 ** 8 if byte < 127 else 2.0 ** -8)
    w13 = torch.zeros(1, 2 * inter, H, dtype=torch.uint8, device="cuda")
    w13[0, 0, 0] = w13[0, inter, 1] = 0x38       # 1: gate 0 = x[0], up 0 = x[1]
    x = torch.zeros(1, H, device="cuda")
    x[0, 0], x[0, 1] = g0, u
    w2 = torch.zeros(1, H, inter, dtype=torch.uint8, device="cuda")
    w2[0, :, 0] = torch.arange(256, dtype=torch.uint8, device="cuda")
    w2[0, 0x7F, 0] = w2[0, 0xFF, 0] = 0          # NaN codes
    n = {M.QUANT_MXFP8: lambda rows: (rows, inter // 32), M.QUANT_FP8_UE8M0: lambda rows: (rows // 128, 4)}[quant]
    put = lambda b, rows: torch.full((1,) + n(rows), b, dtype=torch.uint8, device="cuda").view(  # noqa: E731
        torch.uint8 if quant == M.QUANT_MXFP8 else torch.int32)
    cfg = _cfg(1, H, quant=quant)
    ws = _filled((M.moe_layer_workspace_bytes(cfg, inter),), torch.uint8)
    out = _filled((1, H), torch.bfloat16)
    M.moe_layer_fused(cfg, 1, inter, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                      torch.ones(1, 1, device="cuda"), x.bfloat16(), w13, put(127, 2 * inter), w2, put(byte, H), ws, out)
    torch.cuda.synchronize()
    if byte == 255:
        assert bool(out.isnan().all())
        return
    want = w2[0, :, 0].view(R.F8).double() * 2.0 ** (byte - 127) * (g0 * u)
    assert torch.equal(out[0].double(), want)     # four significant bits: no rounding


@pytest.mark.parametrize("quant", [M.QUANT_FP8_UE8M0, M.QUANT_MXFP8])
@pytest.mark.parametrize("byte", [0, 1, 127, 254, 255])
@pytest.mark.parametrize("T,n", [(1, 256), (130, 256)])
def test_product_weights_at_the_ends_of_their_exponents(T, n, byte, quant):
    _say(f"expert_gemm, exponent byte {byte}, T={T}, quant={quant}")
    k = 128
    a = torch.zeros(T, k, dtype=torch.uint8, device="cuda")
    a[:, 0] = 0x38
    w = torch.zeros(1, n, k, dtype=torch.uint8, device="cuda")
    w[0, :, 0] = torch.arange(256, dtype=torch.uint8, device="cuda")
    w[0, 0x7F, 0] = w[0, 0xFF, 0] = 0
    other = 254 - byte if byte < 255 else 127     # the rows' scale: the product's is 2^0
    put = lambda b, rows: torch.full((rows, 4), b, dtype=torch.uint8, device="cuda").view(  # noqa: E731
        torch.uint8 if quant == M.QUANT_MXFP8 else torch.int32)
    y = _filled((T, n), torch.bfloat16)
    M.moe_expert_gemm(_cfg(T, k, quant=quant), T, n, k, a, put(other, T), w,
                      put(byte, n if quant == M.QUANT_MXFP8 else n // 128)[None], None, y)
    torch.cuda.synchronize()
    if byte == 255:
        assert bool(y.isnan().all())
    else:
        assert torch.equal(y.double(), w[0, :, 0].view(R.F8).double().expand(T, n))


def test_rmsnorm_whose_squares_overflow_gives_zero():
    _say("rmsnorm of 2^64")
    x = torch.ones(2, 256, device="cuda")
    x[0, 3] = 2.0 ** 64
    out, q, _ = _norm(x.bfloat16(), torch.ones(256, device="cuda").bfloat16(), M.QUANT_FP8_F32)
    assert not bool(out[0].any()) and not bool((q[0] & 0x7F).any()) and bool(out[1].all())
