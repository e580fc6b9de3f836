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
from test_gpu_experts import Rows, _cfg, _filled, _gen, _gpu, _layer_reference, _say, _scales  # noqa: F401 (_gpu: a fixture)

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


# ---- kernel variants that need many blocks, rows or channels -------------------------------------------


def _dense_rows(T, k, quant, seed):
    x = torch.randn(T, k, generator=_gen(seed), device="cuda")
    x[::7] *= 100.0
    return R.quantize(x, quant)


def _check_product(y, a, s, w, ws, quant, what):
    """Rows of bf16 against the 64-bit product: each value within its bound, all together within half a step."""
    av = R.dequantize(a, s, quant)
    wv = R.weight_values(w, ws, quant)[0]
    want, bound = R.product(av, wv)
    err = (y.to(D) - want).abs()
    lim = (want.abs() + bound) * 2.0 ** -8 + bound
    assert bool((err <= lim).all()), f"{what}: worst {float((err / lim).max()):.2f} times the bound"
    # a bf16 rounding alone is at most 2^-8 of each value; 2^-15 for the 8-bit products (1.4e-5 measured)
    assert float((y.to(D) - want).norm() / want.norm()) <= 2.0 ** -8 + 2.0 ** -15, what


@pytest.mark.parametrize("quant", FORMATS)
@pytest.mark.parametrize("k", [640, 1024, 1152, 1664])
@pytest.mark.parametrize("T", [2304 + 40, 2304 + 100, 2304 + 200])
def test_products_in_256_row_tiles_of_long_rows(T, k, quant):
    """5, 8, 9 and 13 blocks of channels: the scales' chunks in turn and again, the loop with and without a last
    step; last tiles of at most 64, 128 and 256 rows."""
    n = 6664                                     # 10 row tiles x 27 channel tiles: more than the compute units
    _say(f"expert_gemm T={T} k={k} n={n} quant={quant}")
    a, s = _dense_rows(T, k, quant, T + k)
    w, ws = R.make_weights(_gen(k), 1, n, k, quant, "cuda")
    y = _filled((T + 1, n), torch.bfloat16)
    M.moe_expert_gemm(_cfg(T, k, quant=quant), T, n, k, a, s, w, ws, None, y)
    torch.cuda.synchronize()
    assert bool((y[T:].view(torch.uint8) == 0xA5).all())
    # rows of the first tile, of one inside and of the last
    pick = torch.cat([torch.arange(0, 256, 17, device="cuda"), torch.arange(1280, 1536, 13, device="cuda"),
                      torch.arange(2304, T, 9, device="cuda"), torch.tensor([T - 1], device="cuda")])
    _check_product(y[pick], a[pick], s[pick], w, ws, quant, "picked rows")
    # and all of them against fp32 sums of fp32 products
    wv = R.weight_values(w, ws, quant)[0].float()
    full = R.dequantize(a, s, quant).float() @ wv.T
    assert float((y[:T].float() - full).norm() / full.norm()) <= 2.0 ** -8 + 2.0 ** -15


def _check_swiglu(h, hs, a, s, w, ws, inter, quant, what):
    av = R.dequantize(a, s, quant)
    wv = R.weight_values(w, ws, quant)[0]
    y, bound = R.product(av, wv, eight_bit=quant != M.QUANT_FP8_F32)
    g, u, dg, du = y[:, :inter], y[:, inter:], bound[:, :inter], bound[:, inter:]
    want = R.silu(g) * u
    # |silu'| <= 1.1; the function itself in fp32 (an exponential of argument g: |g| ulps)
    lim = 1.1 * dg * (u.abs() + du) + R.silu(g).abs() * du + want.abs() * (8 + g.abs()) * 2.0 ** -24
    R.assert_rows(h, hs, want, lim, quant, what)
    if quant == M.QUANT_FP8_F32:
        ref = R.block_scale(want.abs().unflatten(-1, (-1, 128)).amax(-1), quant)
        assert float((hs.to(D) - ref).norm() / ref.norm()) <= 1e-5, what
    # E4M3 as a whole: 2^-4 of each value at most (MXFP8 saturates a block's largest by up to 1/8)
    own = R.dequantize(h, hs, quant)
    assert float((own - want).norm() / want.norm()) <= (2.0 ** -3 if quant == M.QUANT_MXFP8 else 2.0 ** -4), what


@pytest.mark.parametrize("quant", FORMATS)
@pytest.mark.parametrize("T,k,inter", [(100, 1152, 256), (45, 1664, 128), (300, 7168, 256), (20, 7168, 128)])
def test_swiglu_of_long_rows(T, k, inter, quant):
    _say(f"expert_gemm_swiglu T={T} k={k} inter={inter} quant={quant}")
    a, s = _dense_rows(T, k, quant, T + k)
    w, ws = R.make_weights(_gen(k), 1, 2 * inter, k, quant, "cuda")
    h, hs = _filled((T, inter), torch.uint8), _scales(T, inter, quant)
    M.moe_expert_gemm_swiglu(_cfg(T, k, quant=quant), T, inter, a, s, w, ws, None, h, hs)
    torch.cuda.synchronize()
    _check_swiglu(h, hs, a, s, w, ws, inter, quant, "all rows")


@pytest.mark.parametrize("quant", FORMATS)
def test_swiglu_of_many_small_tiles_from_memory(quant):
    """Blocks that go from tile to tile, a few rows of another expert each, with caches cold."""
    T, E, K, k, inter = 96, 64, 6, 1024, 2048
    _say(f"expert_gemm_swiglu of many small tiles, caches cold, quant={quant}")
    rows = Rows(15, quant=quant, T=T, E=E, K=K, k=k)
    w, ws = R.make_weights(_gen(16), E, 2 * inter, k, quant, "cuda")
    cold = torch.empty(1 << 29, dtype=torch.uint8, device="cuda")
    h, hs = _filled((rows.rows, inter), torch.uint8), _scales(rows.rows, inter, quant)
    cold.fill_(1)
    M.moe_expert_gemm_swiglu(rows.cfg, T, inter, rows.a, rows.s, w, ws, rows.handle, h, hs)
    torch.cuda.synchronize()
    for e in (0, 13, 21, 42, 63):
        at = slice(rows.off[e], rows.off[e] + rows.count[e])
        _check_swiglu(h[at], hs[at], rows.a[at], rows.s[at], w[e:e + 1], ws[e:e + 1], inter, quant, f"expert {e}")


LAYERS = [
    # 32 channels of h per block (eight blocks per compute unit), one and two groups of 16 tokens
    dict(T=16, E=64, K=4, H=256, inter=1024),
    dict(T=24, E=64, K=4, H=256, inter=1024),
    dict(T=32, E=2, K=1, H=128, inter=32768),    # more than 16 tokens of one expert
    dict(T=40, E=64, K=4, H=256, inter=1024),
    # 32 output channels per block (H past 16 per compute unit), two and four groups
    dict(T=20, E=6, K=2, H=4224, inter=128),
    dict(T=32, E=1, K=1, H=4224, inter=256),
    dict(T=40, E=6, K=2, H=4224, inter=128),
    dict(T=64, E=1, K=1, H=4224, inter=256),
]


@pytest.mark.parametrize("quant", [M.QUANT_NONE] + FORMATS)
@pytest.mark.parametrize("c", LAYERS, ids=lambda c: "T{T}_E{E}_K{K}_H{H}_i{inter}".format(**c))
def test_layer_fused_in_wide_blocks(c, quant):
    _say(f"layer_fused {c} quant={quant}")
    T, E, K, H, inter = c["T"], c["E"], c["K"], c["H"], c["inter"]
    g = _gen(T + E + H)
    idx = torch.topk(torch.rand(T, E, generator=g, device="cuda"), K, 1).indices.to(torch.int32)
    if K > 1:
        idx[3, 1] = -1
        idx[5, 1] = idx[5, 0]
    tw = torch.rand(T, K, generator=g, device="cuda")
    tw[idx < 0] = NAN
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w13, s13 = R.make_weights(g, E, 2 * inter, H, quant, "cuda")
    w2, s2 = R.make_weights(g, E, H, inter, quant, "cuda")
    cfg = _cfg(T, H, E, K, quant)
    ws = _filled((M.moe_layer_workspace_bytes(cfg, inter),), torch.uint8)
    out = _filled((T + 1, H), torch.bfloat16)
    M.moe_layer_fused(cfg, T, inter, idx, tw, x, w13, s13, w2, s2, ws, out)
    torch.cuda.synchronize()
    assert bool((out[T:].view(torch.uint8) == 0xA5).all())
    want, bound = _layer_reference(idx, tw, x, w13, s13, w2, s2, quant, inter)
    err = (out[:T].to(D) - want).abs()
    lim = (want.abs() + bound) * 2.0 ** -8 + bound
    assert bool((err <= lim).all()), float((err / lim).max())
    # both roundings of half a step, as a whole
    assert float((out[:T].to(D) - want).norm()) <= 2.0 ** -7 * float(want.norm())


# ---- weights past 4 GiB --------------------------------------------------------------------------------
# One row of the last expert; the weights of the others are never read (whatever the memory held).


def _last_expert(E, n, k, quant, seed):
    w1, s1 = R.make_weights(_gen(seed), 1, n, k, quant, "cuda")
    w = torch.empty(E, n, k, dtype=torch.uint8, device="cuda")
    s = torch.empty((E,) + tuple(s1.shape[1:]), dtype=s1.dtype, device="cuda")
    w[E - 1], s[E - 1] = w1[0], s1[0]
    return w, s, w1, s1


def _one_row(E, k, quant):
    cfg = _cfg(1, k, E, 1, quant)
    handle = M.Handle(cfg)
    lw = torch.empty(M.moe_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    idx = torch.full((1, 1), E - 1, dtype=torch.int32, device="cuda")
    M.moe_dispatch_layout(cfg, 1, idx, handle, lw)
    a, s = _dense_rows(1, k, quant, k)
    return cfg, handle, idx, a, s


@pytest.mark.parametrize("quant", FORMATS)
def test_strips_read_weights_past_4_gib(quant):
    E, n, k = 2048, 128, 16512                    # 8 strips of 16 channels: fewer than the chip takes at once
    _say(f"expert_gemm, {E * n * k} bytes of weights, the last expert, quant={quant}")
    w, ws, w1, ws1 = _last_expert(E, n, k, quant, 3)
    cfg, handle, _, a, s = _one_row(E, k, quant)
    y = _filled((1, n), torch.bfloat16)
    M.moe_expert_gemm(cfg, 1, n, k, a, s, w, ws, handle, y)
    torch.cuda.synchronize()
    _check_product(y, a, s, w1, ws1, quant, "the last expert")


@pytest.mark.parametrize("quant", FORMATS)
def test_tiles_read_weights_past_4_gib(quant):
    E, n, k = 33, 16384, 8192                     # 1024 strips: 128-row tiles
    _say(f"expert_gemm, {E * n * k} bytes of weights, the last expert, quant={quant}")
    w, ws, w1, ws1 = _last_expert(E, n, k, quant, 4)
    cfg, handle, _, a, s = _one_row(E, k, quant)
    y = _filled((1, n), torch.bfloat16)
    M.moe_expert_gemm(cfg, 1, n, k, a, s, w, ws, handle, y)
    torch.cuda.synchronize()
    _check_product(y, a, s, w1, ws1, quant, "the last expert")


@pytest.mark.parametrize("quant", FORMATS)
def test_swiglu_reads_weights_past_4_gib(quant):
    E, inter, k = 2048, 128, 8320
    _say(f"expert_gemm_swiglu, {E * 2 * inter * k} bytes of weights, the last expert, quant={quant}")
    w, ws, w1, ws1 = _last_expert(E, 2 * inter, k, quant, 5)
    cfg, handle, _, a, s = _one_row(E, k, quant)
    h, hs = _filled((1, inter), torch.uint8), _scales(1, inter, quant)
    M.moe_expert_gemm_swiglu(cfg, 1, inter, a, s, w, ws, handle, h, hs)
    torch.cuda.synchronize()
    _check_swiglu(h, hs, a, s, w1, ws1, inter, quant, "the last expert")


@pytest.mark.parametrize("quant", FORMATS)
def test_layer_reads_weights_past_4_gib(quant):
    E, inter, H = 2048, 256, 8320
    _say(f"layer_fused, {E * inter * H} bytes of w2, the last expert, quant={quant}")
    w13, s13, w13e, s13e = _last_expert(E, 2 * inter, H, quant, 6)
    w2, s2, w2e, s2e = _last_expert(E, H, inter, quant, 7)
    cfg, _, idx, _, _ = _one_row(E, H, quant)
    x = torch.randn(1, H, generator=_gen(8), device="cuda").bfloat16()
    tw = torch.full((1, 1), 0.7, device="cuda")
    ws = _filled((M.moe_layer_workspace_bytes(cfg, inter),), torch.uint8)
    out = _filled((1, H), torch.bfloat16)
    M.moe_layer_fused(cfg, 1, inter, idx, tw, x, w13, s13, w2, s2, ws, out)
    torch.cuda.synchronize()
    want, bound = _layer_reference(torch.zeros_like(idx), tw, x, w13e, s13e, w2e, s2e, quant, inter)
    err = (out.to(D) - want).abs()
    lim = (want.abs() + bound) * 2.0 ** -8 + bound
    assert bool((err <= lim).all()), float((err / lim).max())
    assert float((out.to(D) - want).norm()) <= 2.0 ** -7 * float(want.norm())


@pytest.mark.parametrize("quant", [M.QUANT_NONE] + FORMATS)
@pytest.mark.parametrize("T,E", [(3, 16), (40, 4)])
def test_layer_with_a_token_that_is_not_finite(T, E, quant):
    """NaN or infinity in one token, NaN in another's weights: the other tokens' bytes are as without them."""
    _say(f"layer_fused T={T} E={E}, tokens that are not finite, quant={quant}")
    K, H, inter = 2, 512, 256
    g = _gen(T)
    idx = torch.topk(torch.rand(T, E, generator=g, device="cuda"), K, 1).indices.to(torch.int32)
    tw = torch.rand(T, K, generator=g, device="cuda")
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w13, s13 = R.make_weights(g, E, 2 * inter, H, quant, "cuda")
    w2, s2 = R.make_weights(g, E, H, inter, quant, "cuda")
    cfg = _cfg(T, H, E, K, quant)
    ws = _filled((M.moe_layer_workspace_bytes(cfg, inter),), torch.uint8)

    def run(x, tw):
        out = _filled((T, H), torch.bfloat16)
        M.moe_layer_fused(cfg, T, inter, idx, tw, x, w13, s13, w2, s2, ws, out)
        torch.cuda.synchronize()
        return out

    clean = run(x, tw)
    assert bool(clean.isfinite().all())
    for value in (NAN, INF):
        bad, weights = x.clone(), tw.clone()
        bad[1, 7] = value
        weights[2, 1] = NAN
        got = run(bad, weights)
        rest = [t for t in range(T) if t not in (1, 2)]
        _bytes_equal(got[rest], clean[rest], "another token")
        assert bool(got[2].isnan().all()) and bool((~got[1].isfinite()).any())
