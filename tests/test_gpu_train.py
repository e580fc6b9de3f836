"""The bf16 expert layer and its gradients on the GPU against 64-bit references.

Shapes are small and odd: one row and several hundred, 8 channels and sizes that
end inside a tile, a step or a block of scales, experts without rows, ids that
route nowhere, capacity drops.  Rows without a pair hold NaN and must not be
read; outputs lie in sentinel-filled buffers, and what must not be written is
compared byte for byte.  Bounds come from tests/train_reference.py.

Every test prints the case it runs before touching the GPU.
"""
import pytest
import torch

import combine_topk_idx_amd as M
import train_reference as R

pytestmark = pytest.mark.gpu
D = R.D
SENT = 0xA5
BF16, FP8, UE8M0, MX = M.QUANT_NONE, M.QUANT_FP8_F32, M.QUANT_FP8_UE8M0, M.QUANT_MXFP8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    M.library()


def _say(msg):
    print(f"\n[case] {msg}", flush=True)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _filled(shape, dtype):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.view(torch.uint8).fill_(SENT)
    return t


def _untouched(t, what):
    assert bool((t.contiguous().view(torch.uint8) == SENT).all()), f"{what}: bytes changed that must not"


def _format_buffers(rows, n, quant):
    """Sentinel-filled rows of n channels and their scales (None for bf16)."""
    if quant == BF16:
        return _filled((rows, n), torch.bfloat16), None
    q = _filled((rows, n), torch.uint8)
    if quant == FP8:
        return q, _filled((rows, n // 128), torch.float32)
    if quant == MX:
        return q, _filled((rows, n // 32), torch.uint8)
    return q, _filled((rows, -(-(n // 128) // 4)), torch.int32)


class Rows:
    """A dispatch (or T dense rows, layout None): its config, handle and the rows of every expert."""

    def __init__(self, T, H=8, E=1, K=1, layout=None, align=1, capacity=1, holes=0.0, seed=0, used=None):
        self.T, self.E = T, E
        self.cfg = M.MoeConfig(max_tokens=T + 3, hidden=H, num_experts=E, num_topk=K, num_ranks=1,
                               layout=M.LAYOUT_MASKED if layout == "masked" else M.LAYOUT_CONTIGUOUS, align=align,
                               capacity=capacity)
        if layout is None:
            self.handle, self.n = None, T
            self.spans = [(0, T)]
        else:
            g = _gen(1000 + seed)
            hot = used or E
            score = torch.rand(T, hot, generator=g, device="cuda")
            self.idx = torch.topk(score, min(K, hot), dim=1).indices.to(torch.int32)
            if K > hot:  # the same experts twice
                self.idx = torch.cat([self.idx, self.idx], 1)[:, :K].contiguous()
            if holes:
                self.idx[torch.rand(T, K, generator=g, device="cuda") < holes] = -1
            self.handle = M.Handle(self.cfg)
            ws = torch.empty(max(16, M.moe_workspace_bytes(self.cfg)), dtype=torch.uint8, device="cuda")
            M.moe_dispatch_layout(self.cfg, T, self.idx, self.handle, ws)
            torch.cuda.synchronize()
            self.n = M.moe_rows_capacity(self.cfg)
            off, cnt = self.handle.expert_offset.tolist(), self.handle.recv_count.tolist()
            self.spans = [(off[e], off[e] + cnt[e]) for e in range(E)]
        self.live = torch.zeros(self.n + 2, dtype=torch.bool, device="cuda")
        for lo, hi in self.spans:
            self.live[lo:hi] = True

    def input(self, g, n, std=1.0):
        """bf16 rows with NaN where there is no pair (and in two rows behind the last)."""
        t = (torch.randn(self.n + 2, n, generator=g, device="cuda") * std).bfloat16()
        t[~self.live] = float("nan")
        return t

    def formatted(self, g, n, quant, std=1.0):
        x = self.input(g, n, std)
        if quant == BF16:
            return x, None
        q, s = R.quantize(torch.nan_to_num(x.float()), quant)
        q, s = q.contiguous(), s.contiguous()
        q[~self.live] = 0x7F
        s.view(torch.uint8)[~self.live] = 0xFF
        return q, s

    def values(self, q, s, quant, lo, hi):
        return q[lo:hi].to(D) if quant == BF16 else R.dequantize(q[lo:hi], s[lo:hi], quant)

    def check_untouched(self, t, what):
        if t is not None:
            _untouched(t[~self.live], what)


def _weights(g, *shape):
    return (torch.randn(*shape, generator=g, device="cuda") / shape[-1] ** 0.5).bfloat16()


def _check_saved(rows, q, s, quant, spans_values, what):
    for (lo, hi), (v, b) in spans_values:
        if quant == BF16:
            R.assert_bf16(q[lo:hi], v, b, what)
        else:
            R.assert_rows(q[lo:hi], s[lo:hi], v, b, quant, what)
            if quant == UE8M0 and (v.shape[-1] // 128) % 4:
                assert not bool(s[lo:hi].contiguous().view(torch.uint8)[:, v.shape[-1] // 128:].any())
    rows.check_untouched(q, what)
    rows.check_untouched(s, what + " scales")


LAYOUTS = {
    "one": dict(T=1),
    "dense": dict(T=67),
    "dense300": dict(T=300),
    "dense700": dict(T=700),
    "contiguous": dict(T=41, E=5, K=2, layout="contiguous", align=16, holes=0.2, seed=1),
    "packed": dict(T=90, E=7, K=3, layout="contiguous", align=1, used=4, seed=2),    # experts without rows
    "masked": dict(T=64, E=4, K=2, layout="masked", capacity=21, seed=3),            # drops pairs
    "many": dict(T=700, E=2, K=2, layout="contiguous", align=128, holes=0.1, seed=4),
    "none": dict(T=9, E=3, K=1, layout="contiguous", align=4, holes=1.0, seed=5),    # no pair at all
    "wide": dict(T=150, E=130, K=3, layout="contiguous", align=1, holes=0.1, seed=6),   # few rows of many experts
    "wide_long": dict(T=500, E=129, K=2, layout="contiguous", align=8, used=3, seed=7),  # many rows of few
    # with thousands of channels: 256-row tiles, whose last one is nearly full, half full, a quarter full, one row
    "dense250": dict(T=250),
    "dense340": dict(T=340),
    "dense310": dict(T=310),
    "dense257": dict(T=257),
    "experts": dict(T=300, E=5, K=2, layout="contiguous", align=1, holes=0.1, seed=8),
    "slab": dict(T=260, E=3, K=2, layout="masked", capacity=200, used=2, seed=9),
}


# ---- the gated block ------------------------------------------------------------------


def _run_gated(rows, k, inter, kind, save, seed):
    g = _gen(seed)
    a, w = rows.input(g, k), _weights(g, rows.E, 2 * inter, k)
    h = _filled((rows.n + 2, inter), torch.bfloat16)
    q, s = (None, None) if save is None else _format_buffers(rows.n + 2, 2 * inter, save)
    M.moe_ffn_gated(rows.cfg, rows.T, inter, kind, a, w, rows.handle, h, q, s, BF16 if save is None else save)
    torch.cuda.synchronize()
    return a, w, h, q, s


@pytest.mark.parametrize("layout,k,inter,kind,save", [
    ("one", 8, 8, M.ACT_SILU, None),
    ("one", 7168, 264, M.ACT_SILU, None),
    ("one", 200, 128, M.ACT_GELU, FP8),
    ("one", 64, 136, M.ACT_RELU, BF16),
    ("dense", 72, 24, M.ACT_GELU, None),
    ("dense", 520, 384, M.ACT_SILU, UE8M0),
    ("dense300", 136, 136, M.ACT_NONE, BF16),
    ("dense300", 256, 256, M.ACT_SILU, MX),
    ("dense700", 192, 128, M.ACT_GELU, FP8),
    ("dense700", 328, 200, M.ACT_SILU, BF16),
    ("dense700", 64, 640, M.ACT_SILU, UE8M0),
    ("contiguous", 264, 128, M.ACT_SILU, FP8),
    ("contiguous", 40, 152, M.ACT_RELU, None),
    ("packed", 128, 256, M.ACT_GELU, UE8M0),
    ("packed", 2048, 72, M.ACT_SILU, BF16),
    ("masked", 96, 128, M.ACT_SILU, MX),
    ("many", 136, 384, M.ACT_SILU, MX),
    ("many", 128, 264, M.ACT_GELU, None),
    ("none", 64, 128, M.ACT_SILU, FP8),
    # strips of one expert's rows: 16, 32 and 64 rows
    ("wide", 200, 24, M.ACT_SILU, None),
    ("contiguous", 1096, 24, M.ACT_SILU, BF16),
    ("packed", 584, 40, M.ACT_GELU, BF16),
    # 256-row tiles; one step, odd and even numbers of steps, steps that end early; two rounds over the chip
    ("dense250", 64, 16520, M.ACT_SILU, BF16),
    ("dense250", 328, 49280, M.ACT_SILU, None),
    ("dense340", 8, 12800, M.ACT_GELU, UE8M0),
    ("dense310", 136, 12680, M.ACT_SILU, None),
    ("dense257", 192, 12800, M.ACT_SILU, MX),
    ("experts", 200, 5632, M.ACT_RELU, FP8),
    ("experts", 72, 19720, M.ACT_SILU, BF16),
    ("dense310", 72, 13640, M.ACT_SILU, BF16),
    ("slab", 392, 8448, M.ACT_SILU, UE8M0),
    # 64-row tiles, 256 channels wide, and wider than one round of them: 128 rows
    ("dense257", 136, 384, M.ACT_SILU, UE8M0),
    ("masked", 328, 256, M.ACT_GELU, FP8),
    ("dense", 64, 17024, M.ACT_SILU, MX),
    ("dense300", 72, 7296, M.ACT_SILU, UE8M0),
    # 128-row tiles; the last one nearly full, half full, a quarter full
    ("dense", 72, 16456, M.ACT_GELU, BF16),
    ("dense300", 200, 6728, M.ACT_SILU, BF16),
    ("dense257", 64, 6728, M.ACT_RELU, None),
    ("experts", 392, 3080, M.ACT_SILU, BF16),
    ("slab", 136, 4360, M.ACT_GELU, None),
])
def test_gated(layout, k, inter, kind, save):
    _say(f"gated {layout} k={k} inter={inter} act={kind} save={save}")
    rows = Rows(H=k, **LAYOUTS[layout])
    a, w, h, q, s = _run_gated(rows, k, inter, kind, save, k + inter)
    saved = []
    for e, (lo, hi) in enumerate(rows.spans):
        p, b = R.product(a[lo:hi].to(D), w[e].to(D))
        v, bv = R.gated(p, b, kind)
        R.assert_bf16(h[lo:hi], v, bv, "h")
        saved.append(((lo, hi), (p, b)))
    rows.check_untouched(h, "h")
    if save is not None:
        _check_saved(rows, q, s, save, saved, "saved")


# ---- the product with its epilogue ------------------------------------------------------


@pytest.mark.parametrize("layout,k,n,kind,bias,residual,save", [
    ("one", 8, 8, M.ACT_NONE, False, False, None),
    ("one", 2048, 7168, M.ACT_NONE, True, True, None),
    ("one", 72, 264, M.ACT_SILU, True, False, BF16),
    ("one", 640, 128, M.ACT_GELU, False, True, MX),
    ("dense", 64, 72, M.ACT_RELU, True, True, None),
    ("dense", 136, 640, M.ACT_GELU, True, True, UE8M0),
    ("dense300", 328, 520, M.ACT_GELU, True, True, BF16),
    ("dense300", 64, 256, M.ACT_NONE, False, False, FP8),
    ("dense700", 256, 384, M.ACT_SILU, True, True, FP8),
    ("dense700", 72, 264, M.ACT_NONE, False, True, None),
    ("contiguous", 200, 136, M.ACT_NONE, True, False, None),
    ("contiguous", 64, 128, M.ACT_GELU, True, True, MX),
    ("packed", 1032, 40, M.ACT_SILU, False, False, None),
    ("masked", 128, 264, M.ACT_NONE, True, True, None),
    ("many", 264, 128, M.ACT_RELU, True, True, UE8M0),
    ("many", 64, 1000, M.ACT_NONE, True, False, BF16),
    ("none", 64, 64, M.ACT_NONE, True, True, None),
    # strips of one expert's rows: 16, 32 and 64 rows
    ("wide", 136, 40, M.ACT_GELU, True, True, BF16),
    ("wide", 2120, 8, M.ACT_NONE, True, False, None),
    ("contiguous", 1544, 72, M.ACT_GELU, True, True, BF16),
    ("packed", 584, 24, M.ACT_SILU, True, True, BF16),
    ("masked", 264, 136, M.ACT_RELU, False, True, None),
    # 256-row tiles; one step, odd and even numbers of steps, steps that end early; two rounds over the chip
    ("dense250", 40, 33032, M.ACT_NONE, True, True, BF16),
    ("dense250", 256, 98560, M.ACT_SILU, True, False, None),
    ("dense340", 136, 25608, M.ACT_GELU, True, True, None),
    ("dense310", 200, 25600, M.ACT_SILU, True, True, UE8M0),
    ("dense257", 72, 25600, M.ACT_NONE, True, False, MX),
    ("experts", 392, 11264, M.ACT_GELU, True, True, FP8),
    ("experts", 64, 39432, M.ACT_RELU, True, True, BF16),
    ("dense310", 136, 27144, M.ACT_NONE, True, True, None),
    ("slab", 128, 16904, M.ACT_NONE, True, True, None),
    # 128-row tiles; the last one nearly full, half full, a quarter full
    ("dense", 136, 32904, M.ACT_SILU, True, True, BF16),
    ("dense300", 72, 13448, M.ACT_GELU, True, True, None),
    ("dense257", 264, 13440, M.ACT_SILU, True, True, UE8M0),
    ("experts", 64, 6152, M.ACT_NONE, True, True, BF16),
    ("experts", 200, 6144, M.ACT_GELU, True, False, MX),
    ("slab", 392, 8712, M.ACT_RELU, False, True, None),
    # 64-row tiles past the first round
    ("dense700", 136, 4104, M.ACT_GELU, True, True, BF16),
    ("many", 72, 3080, M.ACT_SILU, True, True, None),
])
def test_linear(layout, k, n, kind, bias, residual, save):
    _say(f"linear {layout} k={k} n={n} act={kind} bias={bias} residual={residual} save={save}")
    rows = Rows(H=8, **LAYOUTS[layout])
    g = _gen(k * 3 + n)
    a, w = rows.input(g, k), _weights(g, rows.E, n, k)
    b = torch.randn(rows.E, n, generator=g, device="cuda").bfloat16() if bias else None
    res = rows.input(g, n, 2.0) if residual else None
    y = _filled((rows.n + 2, n), torch.bfloat16)
    q, s = (None, None) if save is None else _format_buffers(rows.n + 2, n, save)
    M.moe_expert_linear(rows.cfg, rows.T, n, k, kind, a, w, b, res, rows.handle, y, q, s, BF16 if save is None else save)
    torch.cuda.synchronize()
    saved = []
    for e, (lo, hi) in enumerate(rows.spans):
        p, bound = R.product(a[lo:hi].to(D), w[e].to(D))
        if bias:
            p = p + b[e].to(D)
            bound = bound + p.abs() * 2.0 ** -23
        saved.append(((lo, hi), (p, bound)))
        v, _ = R.act(p, kind)
        bv = R.act_bound(p, v, bound, kind)
        if residual:
            v = v + res[lo:hi].to(D)
            bv = bv + v.abs() * 2.0 ** -23
        R.assert_bf16(y[lo:hi], v, bv, "y")
    rows.check_untouched(y, "y")
    if save is not None:
        _check_saved(rows, q, s, save, saved, "saved")


@pytest.mark.parametrize("layout,n", [("one", 256), ("dense", 264), ("dense700", 384), ("contiguous", 72)])
def test_linear_residual_in_place(layout, n):
    _say(f"linear in place {layout} n={n}")
    rows = Rows(**LAYOUTS[layout])
    g = _gen(n)
    a, w, res = rows.input(g, 128), _weights(g, rows.E, n, 128), rows.input(g, n)
    y = _filled(res.shape, torch.bfloat16)
    M.moe_expert_linear(rows.cfg, rows.T, n, 128, M.ACT_SILU, a, w, None, res, rows.handle, y)
    M.moe_expert_linear(rows.cfg, rows.T, n, 128, M.ACT_SILU, a, w, None, res, rows.handle, res)
    torch.cuda.synchronize()
    assert torch.equal(y[rows.live].view(torch.int16), res[rows.live].view(torch.int16))
    assert bool(res[~rows.live].isnan().all())


# ---- the activations' gradients ----------------------------------------------------------


@pytest.mark.parametrize("layout,n,kind,gated,quant,with_y", [
    ("one", 8, M.ACT_SILU, True, BF16, True),
    ("one", 2056, M.ACT_GELU, False, BF16, False),
    ("one", 16384, M.ACT_SILU, True, FP8, True),
    ("dense", 24, M.ACT_GELU, True, BF16, True),
    ("dense", 640, M.ACT_RELU, True, UE8M0, True),
    ("dense300", 136, M.ACT_NONE, True, BF16, True),
    ("dense300", 2176, M.ACT_SILU, False, MX, True),
    ("contiguous", 128, M.ACT_GELU, True, MX, True),
    ("contiguous", 384, M.ACT_GELU, False, FP8, True),
    ("packed", 640, M.ACT_SILU, True, FP8, False),
    ("masked", 128, M.ACT_RELU, False, UE8M0, True),
    ("masked", 520, M.ACT_SILU, True, BF16, True),
    ("none", 128, M.ACT_SILU, True, FP8, True),
])
def test_activation_backward(layout, n, kind, gated, quant, with_y):
    _say(f"activation backward {layout} n={n} act={kind} gated={gated} quant={quant}")
    rows = Rows(**LAYOUTS[layout])
    g = _gen(n + kind)
    m = 2 * n if gated else n
    dy = rows.input(g, n, 0.02)
    q, s = rows.formatted(g, m, quant, 2.0)
    ds = _filled((rows.n + 2, m), torch.bfloat16)
    y = _filled((rows.n + 2, n), torch.bfloat16) if with_y else None
    M.moe_activation_backward(rows.cfg, rows.T, n, kind, gated, dy, q, s, quant, rows.handle, ds, y)
    torch.cuda.synchronize()
    for lo, hi in rows.spans:
        (v, b), (f, bf) = R.act_grads(dy[lo:hi].to(D), rows.values(q, s, quant, lo, hi), kind, gated)
        R.assert_bf16(ds[lo:hi], v, b, "dsaved")
        if with_y:
            R.assert_bf16(y[lo:hi], f, bf, "y")
    rows.check_untouched(ds, "dsaved")
    rows.check_untouched(y, "y")


def test_activation_backward_in_place():
    _say("activation backward into its own arrays")
    rows = Rows(**LAYOUTS["contiguous"])
    g = _gen(7)
    dy, saved = rows.input(g, 72), rows.input(g, 144)
    ds, y = torch.zeros_like(saved), torch.zeros_like(dy)
    args = (rows.cfg, rows.T, 72, M.ACT_SILU, True)
    M.moe_activation_backward(*args, dy, saved, None, BF16, rows.handle, ds, y)
    M.moe_activation_backward(*args, dy, saved, None, BF16, rows.handle, saved, dy)
    torch.cuda.synchronize()
    assert torch.equal(ds[rows.live].view(torch.int16), saved[rows.live].view(torch.int16))
    assert torch.equal(y[rows.live].view(torch.int16), dy[rows.live].view(torch.int16))


@pytest.mark.parametrize("kind", [M.ACT_SILU, M.ACT_GELU, M.ACT_RELU])
def test_activation_backward_far_values(kind):
    """Saved values far from 0 have slopes of 0 or 1, and NaN stays NaN."""
    _say(f"activation backward far values act={kind}")
    far = torch.tensor([-3e38, -1e20, -1e6, -200.0, -100.0, -88.0, -30.0, -0.0, 0.0, 30.0, 88.0, 200.0, 1e6, 1e20, 3e38,
                        1e-40], device="cuda").bfloat16().reshape(1, 16)
    dy = torch.full_like(far, 0.5)
    ds, y = torch.empty_like(far), torch.empty_like(far)
    cfg = M.MoeConfig(max_tokens=1, hidden=8, num_experts=1, num_topk=1, num_ranks=1)
    M.moe_activation_backward(cfg, 1, 16, kind, False, dy, far, None, BF16, None, ds, y)
    v = far.to(D)
    f, s = R.act(v.clamp(-1e6, 1e6), kind)  # the formula in 64 bits, where the cube fits
    f = torch.where(v > 1e6, v, torch.where(v < -1e6, torch.zeros_like(v), f))
    # s = 1 / (1 + exp(-z)) is 0 where 1 + exp(-z) exceeds 2^126 (the hardware's reciprocal has no
    # subnormal results), so f = v s is off by up to |v| 2^-126 there: 5e-37 at -88, where f is 5e-37
    # (1e-38: half a step of bf16's subnormals, for the value 1e-40)
    R.assert_bf16(y, f, 1e-38 + v.abs() * 2.0 ** -126 + f.abs() * 2.0 ** -20, "y")
    R.assert_bf16(ds, 0.5 * s, torch.full_like(f, 2.0 ** -18), "dsaved")
    far[0, 3] = float("nan")
    M.moe_activation_backward(cfg, 1, 16, kind, False, dy, far, None, BF16, None, ds, y)
    torch.cuda.synchronize()
    nan = torch.zeros_like(far, dtype=torch.bool)
    nan[0, 3] = True
    assert torch.equal(ds.isnan(), nan) and torch.equal(y.isnan(), nan)


# ---- the products' gradients ---------------------------------------------------------------


@pytest.mark.parametrize("layout,n,k", [
    ("one", 8, 8), ("one", 264, 2048), ("one", 2056, 136),
    ("dense", 72, 24), ("dense", 64, 256), ("dense", 520, 264),
    ("dense300", 136, 520), ("dense700", 200, 264), ("dense700", 1024, 72),
    ("contiguous", 40, 1000), ("packed", 328, 128), ("masked", 128, 8), ("many", 72, 512), ("none", 64, 64),
    # 256-row tiles; one step, odd and even numbers of steps, steps that end early; two rounds over the chip
    ("dense250", 40, 33032), ("dense250", 136, 98560), ("dense340", 264, 25608), ("dense310", 64, 25600),
    ("dense257", 192, 25600), ("experts", 200, 11272), ("experts", 328, 39432), ("slab", 72, 16904), ("dense310", 200, 27144),
    # 128-row tiles; the last one nearly full, half full, a quarter full
    ("dense", 136, 32904), ("dense300", 72, 13448), ("dense257", 264, 13440), ("experts", 64, 6152), ("slab", 392, 8712),
    # 64-row tiles past the first round
    ("dense700", 136, 4104), ("many", 72, 3080),
])
def test_grad_input(layout, n, k):
    _say(f"grad input {layout} n={n} k={k}")
    rows = Rows(**LAYOUTS[layout])
    g = _gen(n * 5 + k)
    dy, w = rows.input(g, n, 0.02), _weights(g, rows.E, n, k)
    da = _filled((rows.n + 2, k), torch.bfloat16)
    M.moe_expert_grad_input(rows.cfg, rows.T, n, k, dy, w, rows.handle, da)
    torch.cuda.synchronize()
    for e, (lo, hi) in enumerate(rows.spans):
        v, b = R.product(dy[lo:hi].to(D), w[e].to(D).T)
        R.assert_bf16(da[lo:hi], v, b, "da")
    rows.check_untouched(da, "da")


def _grad_weight(rows, n, k, dy, q, s, quant, dw, db, accumulate=False):
    size = M.moe_grad_weight_workspace_bytes(rows.cfg, rows.T, n, k)
    ws = _filled(size, torch.uint8) if size else None
    M.moe_expert_grad_weight(rows.cfg, rows.T, n, k, dy, q, s, quant, rows.handle, dw, db, accumulate, ws)
    torch.cuda.synchronize()


def _grad_weight_reference(rows, dy, q, s, quant):
    for e, (lo, hi) in enumerate(rows.spans):
        d, a = dy[lo:hi].to(D), rows.values(q, s, quant, lo, hi)
        if quant != BF16:
            a = a.float().bfloat16().to(D)  # q * s is exact in 64 bits, and rounds to fp32 before bf16 as the kernel's
        v, b = R.product(d.T, a.T)
        yield e, (v, b), (d.sum(0), (hi - lo + 8) * 2.0 ** -23 * d.abs().sum(0))


@pytest.mark.parametrize("layout,n,k,quant,dtype,bias", [
    ("one", 8, 8, BF16, torch.float32, True),
    ("one", 264, 520, BF16, torch.bfloat16, True),
    ("one", 72, 128, MX, torch.float32, False),
    ("dense", 24, 72, BF16, torch.float32, True),
    ("dense", 256, 256, FP8, torch.bfloat16, False),
    ("dense300", 136, 384, UE8M0, torch.float32, True),
    ("dense700", 520, 264, BF16, torch.bfloat16, True),
    ("dense700", 72, 640, FP8, torch.float32, True),
    ("contiguous", 128, 40, BF16, torch.float32, True),
    ("contiguous", 40, 128, MX, torch.bfloat16, True),
    ("packed", 264, 136, BF16, torch.float32, True),
    ("packed", 136, 256, UE8M0, torch.bfloat16, True),
    ("masked", 200, 128, FP8, torch.float32, True),
    ("many", 328, 264, BF16, torch.float32, True),
    ("many", 64, 384, MX, torch.float32, False),
    ("none", 64, 128, FP8, torch.bfloat16, True),
    # 128 tiles of weights and more: 256 x 256 each
    ("wide", 24, 72, BF16, torch.float32, True),
    ("wide", 264, 40, BF16, torch.bfloat16, True),
    ("wide", 40, 128, FP8, torch.float32, True),
    ("wide_long", 328, 264, BF16, torch.float32, False),
    ("wide_long", 136, 328, BF16, torch.bfloat16, True),
    ("wide_long", 264, 384, FP8, torch.bfloat16, True),
    ("wide_long", 72, 640, UE8M0, torch.float32, True),
    ("wide_long", 264, 256, MX, torch.bfloat16, True),
    ("dense300", 2048, 4096, BF16, torch.float32, True),
    ("dense", 4096, 2048, MX, torch.bfloat16, True),
    ("one", 2056, 4104, BF16, torch.float32, True),
])
def test_grad_weight(layout, n, k, quant, dtype, bias):
    _say(f"grad weight {layout} n={n} k={k} quant={quant} {dtype} bias={bias}")
    rows = Rows(**LAYOUTS[layout])
    g = _gen(n + 7 * k)
    dy = rows.input(g, n, 0.02)
    q, s = rows.formatted(g, k, quant)
    dw = _filled((rows.E + 1, n, k), dtype)
    db = _filled((rows.E + 1, n), torch.float32) if bias else None
    _grad_weight(rows, n, k, dy, q, s, quant, dw, db)
    for e, (v, b), (sv, sb) in _grad_weight_reference(rows, dy, q, s, quant):
        if dtype == torch.float32:
            R.assert_near(dw[e], v, b, f"dw[{e}]")
        else:
            R.assert_bf16(dw[e], v, b, f"dw[{e}]")
        if bias:
            R.assert_near(db[e], sv, sb, f"dbias[{e}]")
    _untouched(dw[rows.E], "dw behind the last expert")
    if bias:
        _untouched(db[rows.E], "dbias behind the last expert")


@pytest.mark.parametrize("layout,n,k", [("dense", 72, 136), ("dense700", 264, 256), ("packed", 40, 264), ("none", 8, 64),
                                        ("wide", 40, 264), ("wide_long", 264, 72)])
def test_grad_weight_accumulates(layout, n, k):
    _say(f"grad weight accumulates {layout} n={n} k={k}")
    rows = Rows(**LAYOUTS[layout])
    g = _gen(n)
    dy, a = rows.input(g, n), rows.input(g, k)
    was = torch.randn(rows.E, n, k, generator=g, device="cuda") * 3
    bwas = torch.randn(rows.E, n, generator=g, device="cuda")
    dw, db = was.clone(), bwas.clone()
    _grad_weight(rows, n, k, dy, a, None, BF16, dw, db, accumulate=True)
    for e, (v, b), (sv, sb) in _grad_weight_reference(rows, dy, a, None, BF16):
        lo, hi = rows.spans[e]
        if lo == hi:
            assert torch.equal(dw[e], was[e]) and torch.equal(db[e], bwas[e])
        R.assert_near(dw[e], was[e].to(D) + v, b + (was[e].to(D).abs() + v.abs()) * 2.0 ** -23, "dw")
        R.assert_near(db[e], bwas[e].to(D) + sv, sb + (bwas[e].to(D).abs() + sv.abs()) * 2.0 ** -23, "dbias")


@pytest.mark.parametrize("T", [64, 65, 511, 4097])
@pytest.mark.parametrize("bias", [False, True])
def test_grad_weight_splits_rows(T, bias):
    """Few weights and many rows: the rows are shared and the parts joined."""
    _say(f"grad weight split T={T} bias={bias}")
    rows = Rows(T)
    g = _gen(T)
    dy, a = rows.input(g, 24), rows.input(g, 72)
    if T == 4097:
        assert M.moe_grad_weight_workspace_bytes(rows.cfg, T, 24, 72) > 0
    for dtype in (torch.float32, torch.bfloat16):
        dw = _filled((2, 24, 72), dtype)
        db = _filled((2, 24), torch.float32) if bias else None
        _grad_weight(rows, 24, 72, dy, a, None, BF16, dw, db)
        for e, (v, b), (sv, sb) in _grad_weight_reference(rows, dy, a, None, BF16):
            (R.assert_near if dtype == torch.float32 else R.assert_bf16)(dw[0], v, b, "dw")
            if bias:
                R.assert_near(db[0], sv, sb, "dbias")
        _untouched(dw[1], "dw")


@pytest.mark.parametrize("quant,accumulate", [(BF16, False), (BF16, True), (FP8, True), (UE8M0, False), (MX, True)])
def test_grad_weight_splits_rows_of_experts(quant, accumulate):
    """Rows shared by several blocks for each of three experts, one of them without rows; dbias with a float's alignment."""
    _say(f"grad weight splits experts' rows quant={quant} accumulate={accumulate}")
    T, n, k = 1700, 72, 256
    rows = Rows(T, E=3, K=2, layout="contiguous", align=16, used=2, holes=0.1, seed=31)
    g = _gen(T)
    dy = rows.input(g, n)
    q, s = rows.formatted(g, k, quant)
    assert M.moe_grad_weight_workspace_bytes(rows.cfg, T, n, k) > 0
    dw, db = torch.randn(4, n, k, generator=g, device="cuda"), torch.randn(3 * n + 2, generator=g, device="cuda")
    was, bwas = dw.clone(), db.clone()
    _grad_weight(rows, n, k, dy, q, s, quant, dw, db[1:-1].view(3, n), accumulate)
    assert torch.equal(dw[3], was[3]) and torch.equal(db[[0, -1]], bwas[[0, -1]])
    for e, (v, b), (sv, sb) in _grad_weight_reference(rows, dy, q, s, quant):
        old, bold = was[e].to(D) * accumulate, bwas[1:-1].view(3, n)[e].to(D) * accumulate
        R.assert_near(dw[e], old + v, b + (old.abs() + v.abs()) * 2.0 ** -23, "dw")
        R.assert_near(db[1:-1].view(3, n)[e], bold + sv, sb + (bold.abs() + sv.abs()) * 2.0 ** -23, "dbias")


def test_grad_weight_of_no_tokens():
    """An empty batch has gradients of zero, or leaves sums as they are."""
    _say("grad weight of no tokens")
    rows = Rows(E=3, K=2, T=5, layout="contiguous")
    dw, db = _filled((3, 16, 24), torch.float32), _filled((3, 16), torch.float32)
    M.moe_expert_grad_weight(rows.cfg, 0, 16, 24, None, None, None, BF16, rows.handle, dw, db, False, None)
    torch.cuda.synchronize()
    assert not bool(dw.any()) and not bool(db.any())
    dw.fill_(2.0)
    M.moe_expert_grad_weight(rows.cfg, 0, 16, 24, None, None, None, BF16, rows.handle, dw, db, True, None)
    torch.cuda.synchronize()
    assert bool((dw == 2.0).all())


# ---- combine's gradient ------------------------------------------------------------------


@pytest.mark.parametrize("T,H,E,K,layout,kw", [
    (1, 8, 1, 1, "contiguous", {}),
    (1, 7168, 8, 8, "contiguous", {}),
    (41, 136, 5, 2, "contiguous", dict(align=16, holes=0.3)),
    (64, 2056, 4, 2, "masked", dict(capacity=21)),
    (13, 520, 2, 4, "contiguous", {}),                         # the same expert twice in one token
    (300, 1024, 16, 3, "masked", dict(capacity=300, holes=0.1)),
    (9, 64, 3, 1, "contiguous", dict(holes=1.0)),
])
def test_combine_backward(T, H, E, K, layout, kw):
    _say(f"combine backward T={T} H={H} E={E} K={K} {layout} {kw}")
    rows = Rows(T, H, E, K, layout, **kw)
    g = _gen(T + H)
    dout = (torch.randn(T, H, generator=g, device="cuda") * 0.02).bfloat16()
    y = rows.input(g, H)
    w = torch.rand(T, K, generator=g, device="cuda") + 0.1
    row = rows.handle.pair_to_row[:T * K].reshape(T, K)
    w[row < 0] = float("nan")                                  # not read
    dy = _filled((rows.n + 2, H), torch.bfloat16)
    dw = _filled((T + 1, K), torch.float32)
    M.moe_combine_backward(rows.cfg, T, dout, y, w, rows.handle, dy, dw)
    torch.cuda.synchronize()
    t, j = torch.nonzero(row >= 0, as_tuple=True)
    at, d = row[t, j].long(), dout[t].to(D)
    v = d * w[t, j].to(D).unsqueeze(1)
    R.assert_bf16(dy[at], v, v.abs() * 2.0 ** -23, "dy")
    yv = y[at].to(D)
    R.assert_near(dw[t, j], (d * yv).sum(1), (H + 8) * 2.0 ** -23 * (d * yv).abs().sum(1), "dtopk_w")
    assert not bool(dw[:T][row < 0].any())
    _untouched(dw[T], "dtopk_w")
    rows.check_untouched(dy, "dy")
    only = _filled(dy.shape, torch.bfloat16)                   # without the weights' gradient, and in place
    M.moe_combine_backward(rows.cfg, T, dout, None, w, rows.handle, only, None)
    M.moe_combine_backward(rows.cfg, T, dout, y, w, rows.handle, y, dw)
    torch.cuda.synchronize()
    assert torch.equal(only.view(torch.int16), dy.view(torch.int16))
    assert torch.equal(y[rows.live].view(torch.int16), dy[rows.live].view(torch.int16))


# ---- used together -------------------------------------------------------------------------


class Layer:
    """A layer's step: dispatch, gated block (saved in 8 bits), down product with biases, combine, and all gradients."""

    def __init__(self, T=150, H=264, E=6, K=2, inter=128, save=UE8M0, seed=11):
        self.T, self.H, self.E, self.K, self.I, self.save = T, H, E, K, inter, save
        self.cfg = M.MoeConfig(max_tokens=T, hidden=H, num_experts=E, num_topk=K, num_ranks=1, align=16)
        g = _gen(seed)
        self.bufs = M.DispatchBuffers(self.cfg)
        n = self.bufs.rows
        self.w13, self.w2 = _weights(g, E, 2 * inter, H), _weights(g, E, H, inter)
        self.bias = (torch.randn(E, H, generator=g, device="cuda") * 0.1).bfloat16()
        new = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        self.h, self.y, self.out = new(n, inter), new(n, H), new(T, H)
        self.saved, self.scale = _format_buffers(n, 2 * inter, save)
        self.dy, self.dtw, self.dh, self.ds, self.h2 = (new(n, H), new(T, K, dt=torch.float32), new(n, inter),
                                                        new(n, 2 * inter), new(n, inter))
        self.dw2, self.db, self.da = new(E, H, inter, dt=torch.float32), new(E, H, dt=torch.float32), new(n, H)
        self.dw13, self.dx, self.ones = new(E, 2 * inter, H), new(T, H), torch.ones(T, K, device="cuda")
        size = max(M.moe_grad_weight_workspace_bytes(self.cfg, T, H, inter),
                   M.moe_grad_weight_workspace_bytes(self.cfg, T, 2 * inter, H), 16)
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        self.x, self.dout = new(T, H), new(T, H)
        self.idx, self.tw = new(T, K, dt=torch.int32), new(T, K, dt=torch.float32)

    def inputs(self, seed):
        g = _gen(seed)
        self.x.copy_(torch.randn(self.T, self.H, generator=g, device="cuda"))
        self.dout.copy_(torch.randn(self.T, self.H, generator=g, device="cuda") * 0.02)
        score = torch.rand(self.T, self.E, generator=g, device="cuda")
        w, idx = torch.topk(score, self.K, dim=1)
        self.idx.copy_(idx)
        self.tw.copy_(w / w.sum(1, keepdim=True))

    def step(self):
        c, T, H, I, b = self.cfg, self.T, self.H, self.I, self.bufs
        i16 = lambda t: t.view(torch.int16)  # noqa: E731
        M.moe_dispatch_fused(c, T, self.idx, i16(self.x), None, b.handle, b.workspace, b.out_x)
        M.moe_ffn_gated(c, T, I, M.ACT_SILU, b.out_x, self.w13, b.handle, self.h, self.saved, self.scale, self.save)
        M.moe_expert_linear(c, T, H, I, M.ACT_NONE, self.h, self.w2, self.bias, None, b.handle, self.y)
        M.moe_combine(c, T, i16(self.y), self.tw, b.handle, i16(self.out))
        M.moe_combine_backward(c, T, self.dout, self.y, self.tw, b.handle, self.dy, self.dtw)
        M.moe_expert_grad_input(c, T, H, I, self.dy, self.w2, b.handle, self.dh)
        M.moe_activation_backward(c, T, I, M.ACT_SILU, True, self.dh, self.saved, self.scale, self.save, b.handle, self.ds,
                                  self.h2)
        M.moe_expert_grad_weight(c, T, H, I, self.dy, self.h2, None, BF16, b.handle, self.dw2, self.db, False, self.ws)
        M.moe_expert_grad_input(c, T, 2 * I, H, self.ds, self.w13, b.handle, self.da)
        M.moe_expert_grad_weight(c, T, 2 * I, H, self.ds, b.out_x, None, BF16, b.handle, self.dw13, None, False, self.ws)
        M.moe_combine(c, T, i16(self.da), self.ones, b.handle, i16(self.dx))

    def outputs(self):
        return {k: getattr(self, k).clone() for k in ("out", "dtw", "dw2", "db", "dw13", "dx")}


def _loss(layer, x, w13, w2, bias, tw):
    """<dout, layer(x)> in 64 bits."""
    total = 0.0
    for e in range(layer.E):
        t, j = torch.nonzero(layer.idx == e, as_tuple=True)
        g, u = (x[t] @ w13[e].T).chunk(2, -1)
        y = (g * torch.sigmoid(g) * u) @ w2[e].T + bias[e]
        total = total + (y * tw[t, j].unsqueeze(1) * layer.dout.to(D)[t]).sum()
    return total


@pytest.mark.parametrize("save", [BF16, FP8, UE8M0, MX])
def test_layer_gradients_against_differences(save):
    """Every gradient of a step against central differences of the 64-bit loss, along random
    directions and along the gradient itself.

    An intermediate rounded to bf16 is off by 2^-9 of itself at most; five lie between a
    gradient and the loss (h, y or dy, dh, dsaved, the result), and their errors are
    independent, so that along a direction with N terms they add up as roots: allowed is
    5 * 2^-8 of the root of the sum of squares, times 4 (four standard deviations).  Rows
    saved in 8 bits are off by 2^-4 of themselves, which passes to the gradients behind
    them with a factor of at most 2 (slope and value both use it).
    """
    _say(f"layer gradients save={save}")
    L = Layer(save=save)
    L.inputs(21)
    L.step()
    torch.cuda.synchronize()
    got = L.outputs()
    base = dict(x=L.x.to(D), w13=L.w13.to(D), w2=L.w2.to(D), bias=L.bias.to(D), tw=L.tw.to(D))
    grads = dict(x=got["dx"], w13=got["dw13"], w2=got["dw2"], bias=got["db"], tw=got["dtw"])
    g = _gen(5)
    for name, grad in grads.items():
        eight = 2.0 ** -4 * 2 if save != BF16 and name in ("x", "w13", "w2") else 0.0
        for trial in range(3):
            d = torch.randn(base[name].shape, generator=g, device="cuda", dtype=D)
            if trial == 0:
                d = grad.to(D) / grad.to(D).norm() * d.norm()
            h = 1e-5
            plus, minus = (_loss(L, **{**base, name: base[name] + s * h * d}) for s in (1, -1))
            diff = float((plus - minus) / (2 * h))
            terms = grad.to(D) * d
            allowed = (5 * 2.0 ** -8 + eight) * 4 * float(terms.norm()) + 1e-6
            if trial == 0:  # along the gradient errors of one sign do not cancel as roots
                allowed += (5 * 2.0 ** -9 + eight / 2) * float(terms.abs().sum())
            assert abs(float(terms.sum()) - diff) <= allowed, (name, trial, float(terms.sum()), diff, allowed)


def test_layer_in_a_graph():
    """A step captured once and replayed on changed inputs, with eager work in between: every replay as eager."""
    _say("layer in a graph")
    L = Layer()
    L.inputs(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        L.step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.step()
    for seed in (2, 3, 2, 4):
        L.inputs(seed)
        graph.replay()
        torch.cuda.synchronize()
        replayed = L.outputs()
        L.step()
        torch.cuda.synchronize()
        for k, v in L.outputs().items():
            assert torch.equal(replayed[k], v), (seed, k)


def test_layers_on_two_streams():
    """Two layers' steps at once give what each gives alone."""
    _say("layers on two streams")
    a, b = Layer(seed=1), Layer(T=90, H=136, E=4, K=3, inter=256, save=MX, seed=2)
    want = []
    for i, L in enumerate((a, b)):
        L.inputs(30 + i)
        L.step()
        torch.cuda.synchronize()
        want.append(L.outputs())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, L in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                L.step()
    torch.cuda.synchronize()
    for L, w in zip((a, b), want):
        for k, v in L.outputs().items():
            assert torch.equal(w[k], v), k


def test_explicit_stream_and_device():
    _say("explicit stream")
    cfg = M.MoeConfig(max_tokens=33, hidden=64, num_experts=1, num_topk=1, num_ranks=1)
    g = _gen(1)
    dy, w = torch.randn(33, 64, generator=g, device="cuda").bfloat16(), _weights(g, 1, 64, 64)
    out, ref = torch.zeros_like(dy), torch.zeros_like(dy)
    M.moe_expert_grad_input(cfg, 33, 64, 64, dy, w, None, ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    M.moe_expert_grad_input(cfg, 33, 64, 64, dy, w, None, out, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    for bad in (dy.cpu(), dy[:, :32], dy.float()):
        with pytest.raises(ValueError):
            M.moe_expert_grad_input(cfg, 33, 64, 64, bad, w, None, out)
    with pytest.raises(ValueError):
        M.moe_ffn_gated(cfg, 33, 32, M.ACT_SILU, dy, w, None, out, None, out)     # scales without rows
    with pytest.raises(ValueError):
        M.moe_expert_grad_input(cfg, 33, 64, 64, dy, w[:, :32], None, out)
    with pytest.raises(M.MoeError):
        M.moe_expert_linear(cfg, 33, 64, 64, 9, dy, w, None, None, None, out)


# ---- values that are not finite -----------------------------------------------------------


@pytest.mark.parametrize("T", [3, 40, 600])
def test_rows_do_not_mix(T):
    """NaN and infinities of one row, channel or expert show nowhere else."""
    _say(f"rows do not mix T={T}")
    rows = Rows(T, H=136, E=3, K=2, layout="contiguous", align=8, seed=9)
    g = _gen(T)
    a, w = rows.input(g, 136), _weights(g, 3, 128, 136)
    lo, hi = next(s for s in rows.spans if s[1] - s[0] > 1)
    bad = lo + (hi - lo) // 2
    y = [torch.zeros(rows.n + 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    hh = [torch.zeros(rows.n + 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    da = [torch.zeros(rows.n + 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dw = [torch.zeros(3, 136, 128, device="cuda") for _ in range(2)]
    w2 = _weights(g, 3, 136, 128)
    x128 = rows.input(g, 128)
    for i in range(2):
        if i:
            a[bad, 5], a[bad, 130] = float("nan"), float("inf")
        M.moe_expert_linear(rows.cfg, T, 128, 136, M.ACT_SILU, a, w, None, None, rows.handle, y[i])
        M.moe_ffn_gated(rows.cfg, T, 64, M.ACT_GELU, a, w, rows.handle, hh[i])
        M.moe_expert_grad_input(rows.cfg, T, 136, 128, a, w2, rows.handle, da[i])
        size = M.moe_grad_weight_workspace_bytes(rows.cfg, T, 136, 128)
        ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
        M.moe_expert_grad_weight(rows.cfg, T, 136, 128, a, x128, None, BF16, rows.handle, dw[i], None, False, ws)
    torch.cuda.synchronize()
    for was, now in (y, hh, da):
        keep = rows.live.clone()
        keep[bad] = False
        assert torch.equal(was[keep], now[keep])
        assert bool(now[bad].isnan().all())
    e = next(i for i, s in enumerate(rows.spans) if s == (lo, hi))
    nan = dw[1].isnan()
    assert bool(nan[e, 5].all()) and bool((nan[e, 130] | dw[1][e, 130].isinf()).all())
    nan[e, 5], nan[e, 130] = False, False
    assert not bool(nan.any())
    dw[0][e, [5, 130]], dw[1][e, [5, 130]] = 0.0, 0.0
    assert torch.equal(*dw)


@pytest.mark.parametrize("T", [3, 600])
@pytest.mark.parametrize("save", [FP8, UE8M0, MX])
def test_saved_rows_do_not_mix(T, save):
    """A row with a NaN is saved as NaN in 8 bits, and no other row shows it."""
    _say(f"saved rows do not mix T={T} save={save}")
    rows = Rows(T, H=136, E=3, K=2, layout="contiguous", align=8, seed=9)
    g = _gen(T)
    a, w = rows.input(g, 136), _weights(g, 3, 512, 136)
    lo, hi = next(s for s in rows.spans if s[1] - s[0] > 1)
    bad = lo + (hi - lo) // 2
    got = []
    for i in range(2):
        if i:
            a[bad, 5] = float("nan")
        y, h = _filled((rows.n, 512), torch.bfloat16), _filled((rows.n, 256), torch.bfloat16)
        (q, s), (gq, gs) = _format_buffers(rows.n, 512, save), _format_buffers(rows.n, 512, save)
        M.moe_expert_linear(rows.cfg, T, 512, 136, M.ACT_SILU, a, w, None, None, rows.handle, y, q, s, save)
        M.moe_ffn_gated(rows.cfg, T, 256, M.ACT_SILU, a, w, rows.handle, h, gq, gs, save)
        got.append([y, h, q, s, gq, gs])
    torch.cuda.synchronize()
    keep = torch.arange(rows.n, device="cuda") != bad
    for was, now in zip(*got):
        assert torch.equal(was[keep].view(torch.uint8), now[keep].view(torch.uint8))
    y, h, q, _, gq, _ = got[1]
    assert bool(y[bad].isnan().all()) and bool(h[bad].isnan().all())
    assert bool(((q[bad] & 0x7F) == 0x7F).all()) and bool(((gq[bad] & 0x7F) == 0x7F).all())


# ---- many experts -------------------------------------------------------------------------


def test_most_experts():
    """2048 experts of a few rows each, and the most choices of a token."""
    _say("2048 experts")
    T, E, K, k, n = 90, 2048, 32, 72, 128
    rows = Rows(T, H=k, E=E, K=K, layout="contiguous", align=4, holes=0.1, seed=41)
    g = _gen(41)
    a, w, dy = rows.input(g, k), _weights(g, E, n, k), rows.input(g, n)
    y, z = _filled((rows.n + 2, n), torch.bfloat16), _filled((rows.n + 2, n), torch.bfloat16)
    h, da = _filled((rows.n + 2, n // 2), torch.bfloat16), _filled((rows.n + 2, k), torch.bfloat16)
    q, s = _format_buffers(rows.n + 2, n, UE8M0)
    dw, db = _filled((E, n, k), torch.float32), _filled((E, n), torch.float32)
    M.moe_expert_linear(rows.cfg, T, n, k, M.ACT_NONE, a, w, None, None, rows.handle, y)
    M.moe_expert_linear(rows.cfg, T, n, k, M.ACT_NONE, a, w, None, None, rows.handle, z, q, s, UE8M0)
    M.moe_ffn_gated(rows.cfg, T, n // 2, M.ACT_SILU, a, w, rows.handle, h)
    M.moe_expert_grad_input(rows.cfg, T, n, k, dy, w, rows.handle, da)
    _grad_weight(rows, n, k, dy, a, None, BF16, dw, db)
    expert = torch.full((rows.n,), -1, device="cuda")
    for e, (lo, hi) in enumerate(rows.spans):
        expert[lo:hi] = e
    at = torch.nonzero(expert >= 0).squeeze(1)
    of = expert[at]
    for e0 in range(0, E, 512):  # 64-bit weights of a share of the experts
        some = at[(of >= e0) & (of < e0 + 512)]
        we = w[expert[some]].to(D)
        x, d = a[some].to(D), dy[some].to(D)
        p = (we * x.unsqueeze(1)).sum(2)
        b = (k + 8) * 2.0 ** -23 * (we * x.unsqueeze(1)).abs().sum(2)
        R.assert_bf16(y[some], p, b, "y")
        R.assert_bf16(z[some], p, b, "y beside saved rows")
        R.assert_rows(q[some], s[some], p, b, UE8M0, "saved")
        v, bv = R.gated(p, b, R.SILU)
        R.assert_bf16(h[some], v, bv, "h")
        v = (we * d.unsqueeze(2)).sum(1)
        R.assert_bf16(da[some], v, (n + 8) * 2.0 ** -23 * (we * d.unsqueeze(2)).abs().sum(1), "da")
        want, bound = torch.zeros(512, n, k, dtype=D, device="cuda"), torch.zeros(512, n, k, dtype=D, device="cuda")
        terms = d.unsqueeze(2) * x.unsqueeze(1)
        want.index_add_(0, expert[some] - e0, terms)
        bound.index_add_(0, expert[some] - e0, terms.abs())
        R.assert_near(dw[e0:e0 + 512], want, bound * (T + 8) * 2.0 ** -23, "dw")
        bias, size = torch.zeros(512, n, dtype=D, device="cuda"), torch.zeros(512, n, dtype=D, device="cuda")
        bias.index_add_(0, expert[some] - e0, d)
        size.index_add_(0, expert[some] - e0, d.abs())
        R.assert_near(db[e0:e0 + 512], bias, size * (T + 8) * 2.0 ** -23, "dbias")
    for t, what in ((y, "y"), (z, "y beside saved rows"), (q, "saved"), (s, "scales"), (h, "h"), (da, "da")):
        rows.check_untouched(t, what)


# ---- offsets past 32 bits -----------------------------------------------------------------


def test_rows_past_4_gib():
    """More than 2^32 bytes of rows, in every operator that addresses rows."""
    _say("rows past 4 GiB")
    T, k, n = 33025, 65544, 8   # 4.3 GB of bf16
    cfg = M.MoeConfig(max_tokens=T, hidden=k, num_experts=1, num_topk=1, num_ranks=1)
    a = torch.zeros(T, k, dtype=torch.bfloat16, device="cuda")
    g = _gen(1)
    at = [0, 127, 16384, 32768, T - 2, T - 1]
    a[at] = torch.randn(len(at), k, generator=g, device="cuda").bfloat16()
    w = _weights(g, 1, n, k)
    y = torch.empty(T, n, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_linear(cfg, T, n, k, M.ACT_NONE, a, w, None, None, None, y)
    v, b = R.product(a[at].to(D), w[0].to(D))
    R.assert_bf16(y[at], v, b, "y")
    dw = torch.empty(1, n, k, device="cuda")
    size = M.moe_grad_weight_workspace_bytes(cfg, T, n, k)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    dy = torch.ones(T, n, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_grad_weight(cfg, T, n, k, dy, a, None, BF16, None, dw, None, False, ws)
    R.assert_near(dw[0, 3], a[at].to(D).sum(0), a[at].to(D).abs().sum(0) * 16 * 2.0 ** -23, "dw")
    del ws
    out = torch.empty_like(a)
    M.moe_expert_grad_input(cfg, T, n, k, y, w, None, out)
    v, b = R.product(y[at].to(D), w[0].to(D).T)
    R.assert_bf16(out[at], v, b, "da")
    M.moe_activation_backward(cfg, T, k, M.ACT_SILU, False, out, a, None, BF16, None, a, out)
    assert bool(a[at].any(1).all()) and bool(out[T - 1].any())
    torch.cuda.synchronize()


def test_weights_past_4_gib():
    """Weights and their gradients past 2^32 bytes."""
    _say("weights past 4 GiB")
    E, n, k = 40, 4096, 8200
    rows = Rows(5, H=k, E=E, K=8, layout="contiguous", seed=3)
    g = _gen(2)
    w = torch.zeros(E, n, k, dtype=torch.bfloat16, device="cuda")
    e = max(i for i, (lo, hi) in enumerate(rows.spans) if hi > lo)
    assert e > 32
    w[e] = _weights(g, n, k)
    lo, hi = rows.spans[e]
    a = rows.input(g, k)
    y = torch.zeros(rows.n + 2, n, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_linear(rows.cfg, 5, n, k, M.ACT_NONE, a, w, None, None, rows.handle, y)
    v, b = R.product(a[lo:hi].to(D), w[e].to(D))
    R.assert_bf16(y[lo:hi], v, b, "y")
    h = torch.zeros(rows.n + 2, n // 2, dtype=torch.bfloat16, device="cuda")
    M.moe_ffn_gated(rows.cfg, 5, n // 2, M.ACT_SILU, a, w, rows.handle, h)
    R.assert_bf16(h[lo:hi], *R.gated(v, b, R.SILU), "h")
    da = torch.zeros(rows.n + 2, k, dtype=torch.bfloat16, device="cuda")
    M.moe_expert_grad_input(rows.cfg, 5, n, k, y, w, rows.handle, da)
    R.assert_bf16(da[lo:hi], *R.product(y[lo:hi].to(D), w[e].to(D).T), "da")
    del w
    dw = _filled((E, n, k), torch.float32)  # 5.4 GB
    size = M.moe_grad_weight_workspace_bytes(rows.cfg, 5, n, k)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    M.moe_expert_grad_weight(rows.cfg, 5, n, k, y, a, None, BF16, rows.handle, dw, None, False, ws)
    v, b = R.product(y[lo:hi].to(D).T, a[lo:hi].to(D).T)
    R.assert_near(dw[e], v, b, "dw")
    empty = [i for i, (p, q) in enumerate(rows.spans) if p == q]
    assert empty and not bool(dw[empty[-1]].any())
    torch.cuda.synchronize()
