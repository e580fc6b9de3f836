"""The expert-layer operators on the GPU against 64-bit references.

Shapes are small and odd: one token and several hundred, one 128-channel block
and many, row groups that end inside a tile, experts without rows, ids that
route nowhere, capacity drops, rows and scales holding NaN where no pair is.
Outputs lie in sentinel-filled buffers, and what must not be written is compared
byte for byte.  Bounds come from tests/expert_reference.py.

Every test prints the case it runs before touching the GPU.
"""
import pytest
import torch

import combine_topk_idx_amd as M
import expert_reference as R

pytestmark = pytest.mark.gpu
D = R.D
FORMATS = [M.QUANT_FP8_F32, M.QUANT_FP8_UE8M0, M.QUANT_MXFP8]
SENT = 0xA5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    M.library()


def _say(msg):
    print(f"\n[case] {msg}", flush=True)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _cfg(T, H, E=1, K=1, quant=M.QUANT_FP8_F32, layout=M.LAYOUT_CONTIGUOUS, align=1, capacity=1):
    return M.MoeConfig(max_tokens=T, hidden=H, num_experts=E, num_topk=K, num_ranks=1, layout=layout, align=align,
                       capacity=capacity, quant=quant)


def _filled(shape, dtype):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.view(torch.uint8).fill_(SENT)
    return t


def _scales(rows, n, quant):
    if quant == M.QUANT_FP8_F32:
        return _filled((rows, n // 128), torch.float32)
    if quant == M.QUANT_MXFP8:
        return _filled((rows, n // 32), torch.uint8)
    return _filled((rows, -(-(n // 128) // 4)), torch.int32)


def _untouched(t, what):
    assert bool((t.contiguous().view(torch.uint8) == SENT).all()), f"{what}: bytes changed that must not"


# ---- norm ------------------------------------------------------------------------------


@pytest.mark.parametrize("T,H,quant,residual,out,rows", [
    (1, 128, M.QUANT_FP8_F32, True, True, True),
    (1, 7168, M.QUANT_FP8_UE8M0, True, True, True),
    (3, 136, M.QUANT_NONE, True, True, False),         # a row that ends inside a wave's second load
    (5, 8, M.QUANT_NONE, False, True, False),
    (7, 640, M.QUANT_FP8_UE8M0, False, False, True),   # five blocks: three unused scale bytes
    (257, 2048, M.QUANT_MXFP8, True, True, True),
    (258, 2176, M.QUANT_FP8_F32, False, True, True),
    (33, 8192, M.QUANT_MXFP8, True, False, True),
    (9, 8320, M.QUANT_FP8_UE8M0, True, True, True),
    (2, 32768, M.QUANT_FP8_F32, True, True, True),
    (1025, 256, M.QUANT_FP8_F32, True, True, False),
])
def test_rmsnorm(T, H, quant, residual, out, rows):
    _say(f"rmsnorm T={T} H={H} quant={quant} residual={residual} out={out} rows={rows}")
    g = _gen(T * 7 + H)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    x[T // 2] *= 2.0 ** -30 if T > 1 else 1.0   # a row far below the others
    res = (torch.randn(T, H, generator=g, device="cuda") * 3).bfloat16() if residual else None
    w = torch.randn(H, generator=g, device="cuda").bfloat16()
    eps = 1e-6
    cfg = _cfg(T, H, quant=quant)
    n = T + 2  # two rows past the last: left as they were
    o = _filled((n, H), torch.bfloat16) if out else None
    ro = _filled((n, H), torch.bfloat16) if residual else None
    q = _filled((n, H), torch.uint8) if rows else None
    s = _scales(n, H, quant) if rows else None
    M.moe_rmsnorm(cfg, T, x, res, w, eps, ro, o, q, s)
    torch.cuda.synchronize()
    r = x.float()
    if residual:
        r = (r + res.float()).bfloat16()
        assert torch.equal(ro[:T].view(torch.int16), r.view(torch.int16))
        _untouched(ro[T:], "residual_out")
    r = r.to(D)
    y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * w.to(D)
    # the sum (H terms), mean, root, reciprocal and two products in fp32
    bound = y.abs() * (H + 8) * 2.0 ** -24
    if out:
        R.assert_bf16(o[:T], y, bound, "out")
        _untouched(o[T:], "out")
    if rows:
        R.assert_rows(q[:T], s[:T], y, bound, quant, "rows")
        if quant == M.QUANT_FP8_UE8M0 and (H // 128) % 4:
            assert not bool(s[:T].view(torch.uint8)[:, H // 128:].any())
        _untouched(q[T:], "out_q")
        _untouched(s[T:], "out_scale")


def test_rmsnorm_in_place():
    _say("rmsnorm with residual_out = residual and out = x")
    T, H = 19, 1024
    g = _gen(3)
    x, res = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.ones(H, device="cuda").bfloat16()
    cfg = _cfg(T, H)
    a = [torch.empty_like(x), torch.empty_like(x)]
    M.moe_rmsnorm(cfg, T, x, res, w, 1e-5, a[0], a[1])
    xi, ri = x.clone(), res.clone()
    M.moe_rmsnorm(cfg, T, xi, ri, w, 1e-5, ri, xi)
    torch.cuda.synchronize()
    assert torch.equal(ri, a[0]) and torch.equal(xi, a[1])


# ---- products -----------------------------------------------------------------------------


class Rows:
    """Dispatched rows of a random routing: E4M3 rows and scales, NaN where no pair is, and the handle."""

    def __init__(self, seed, T, E, K, k, quant, layout="contiguous", align=1, capacity=1, holes=0.0, skew=0.0):
        g = _gen(seed)
        self.T, self.E, self.k, self.quant = T, E, k, quant
        self.handle = None
        if layout == "dense":
            self.cfg = _cfg(T, k, quant=quant)
            self.rows, self.off, self.count = T, [0], [T]
        else:
            score = torch.rand(T, E, generator=g, device="cuda") - skew * torch.arange(E, device="cuda") / E
            idx = torch.topk(score, K, 1).indices.to(torch.int32)
            if holes:
                idx[torch.rand(T, K, generator=g, device="cuda") < holes] = -1
                idx[0, 0] = E + 5  # an invalid id
            self.cfg = _cfg(T, k, E, K, quant, M.LAYOUT_MASKED if layout == "masked" else M.LAYOUT_CONTIGUOUS, align,
                            capacity)
            self.idx = idx.contiguous()
            self.handle = M.Handle(self.cfg)
            ws = torch.empty(M.moe_workspace_bytes(self.cfg), dtype=torch.uint8, device="cuda")
            M.moe_dispatch_layout(self.cfg, T, self.idx, self.handle, ws)
            self.rows = M.moe_rows_capacity(self.cfg)
            self.off = self.handle.expert_offset[:E].tolist()
            self.count = self.handle.recv_count.tolist()
        x = torch.randn(self.rows, k, generator=g, device="cuda")
        x[:: 7] *= 100.0
        self.a, self.s = R.quantize(x, quant)
        self.used = torch.zeros(self.rows, dtype=torch.bool, device="cuda")
        for o, c in zip(self.off, self.count):
            self.used[o:o + c] = True
        self.a[~self.used] = 0x7F  # E4M3 NaN
        if quant == M.QUANT_FP8_F32:
            self.s[~self.used] = float("nan")
        else:
            self.s.view(torch.uint8)[~self.used] = 255


CASES = [
    # few rows per expert
    dict(T=1, E=4, K=1, k=128, n=8),
    dict(T=3, E=5, K=2, k=256, n=256),
    dict(T=40, E=16, K=2, k=640, n=264, layout="masked", capacity=3),          # drops
    dict(T=64, E=8, K=2, k=384, n=520, align=16, holes=0.3),
    dict(T=100, E=64, K=4, k=256, n=104, skew=2.0, align=8),                   # one expert with many rows
    dict(T=7, E=1, K=1, k=1024, n=72, layout="dense"),
    # 128-row tiles
    dict(T=130, E=2, K=2, k=128, n=256, align=128),
    dict(T=300, E=4, K=2, k=896, n=392, holes=0.2),
    dict(T=257, E=3, K=1, k=512, n=128, layout="masked", capacity=200, skew=3.0),
    dict(T=1111, E=1, K=1, k=256, n=776, layout="dense"),
    dict(T=161, E=6, K=5, k=1408, n=256, align=32),
    dict(T=129, E=1, K=1, k=128, n=16, layout="dense"),
    # 256-row tiles: enough of them for every compute unit
    dict(T=2309, E=1, K=1, k=384, n=8200, layout="dense"),
    dict(T=1300, E=2, K=1, k=256, n=16384, align=128),
    # few rows, more 16-channel strips than the chip takes at once
    dict(T=1, E=1, K=1, k=128, n=10264, layout="dense"),
    dict(T=3, E=5, K=2, k=256, n=4104),
    dict(T=40, E=16, K=2, k=640, n=776, layout="masked", capacity=3),
    dict(T=100, E=64, K=4, k=256, n=520, skew=2.0, align=8),
    dict(T=257, E=3, K=1, k=512, n=1288, layout="masked", capacity=200, skew=3.0),
    # few strips: many rows of few channels, long rows
    dict(T=2000, E=3, K=2, k=384, n=24, align=16),
    dict(T=16, E=1, K=1, k=5120, n=264, layout="dense"),
    # many experts, most without rows, their number no multiple of the table's groups
    dict(T=60, E=2047, K=1, k=128, n=264),
    dict(T=60, E=2047, K=1, k=128, n=8),
]


@pytest.mark.parametrize("quant", FORMATS)
@pytest.mark.parametrize("case", CASES, ids=lambda c: "T{T}_E{E}_K{K}_k{k}_n{n}".format(**c))
def test_expert_gemm(case, quant):
    _say(f"expert_gemm {case} quant={quant}")
    c = dict(case)
    n = c.pop("n")
    rows = Rows(c["T"] * 13 + n, quant=quant, **c)
    w, ws = R.make_weights(_gen(n + c["k"]), rows.E, n, c["k"], quant, "cuda")
    y = _filled((rows.rows, n), torch.bfloat16)
    M.moe_expert_gemm(rows.cfg, c["T"], n, c["k"], rows.a, rows.s, w, ws, rows.handle, y)
    torch.cuda.synchronize()
    _untouched(y[~rows.used], "rows without a pair")
    for e, (o, m) in enumerate(zip(rows.off, rows.count)):
        if m == 0:
            continue
        a = R.dequantize(rows.a[o:o + m], rows.s[o:o + m], quant)
        wv = R.weight_values(w[e:e + 1], ws[e:e + 1], quant)[0]
        pick = torch.arange(m, device="cuda") if m <= 320 else torch.cat(  # ends and borders of the tiles
            [torch.arange(260, device="cuda"), torch.arange(m - 40, m, device="cuda")])
        want, bound = R.product(a[pick], wv)
        R.assert_bf16(y[o:o + m][pick], want, bound, f"expert {e}")
        got = y[o:o + m].to(D)
        full = a @ wv.T
        # half a bf16 step per value, and 2^-15 for the 8-bit products (1.4e-5 measured)
        assert float((got - full).norm() / full.norm()) <= 2.0 ** -8 + 2.0 ** -15


SWIGLU = [
    dict(T=1, E=4, K=1, k=128, inter=128),
    dict(T=5, E=8, K=3, k=256, inter=640),
    dict(T=64, E=8, K=2, k=256, inter=128, holes=0.2),
    dict(T=70, E=32, K=2, k=640, inter=256, layout="masked", capacity=4),
    dict(T=200, E=3, K=2, k=384, inter=384, align=128),
    dict(T=333, E=1, K=1, k=512, inter=128, layout="dense"),
    dict(T=1500, E=1, K=1, k=256, inter=8192, layout="dense"),
]


@pytest.mark.parametrize("quant", FORMATS)
@pytest.mark.parametrize("case", SWIGLU, ids=lambda c: "T{T}_E{E}_K{K}_k{k}_i{inter}".format(**c))
def test_expert_gemm_swiglu(case, quant):
    _say(f"expert_gemm_swiglu {case} quant={quant}")
    c = dict(case)
    inter = c.pop("inter")
    rows = Rows(c["T"] * 11 + inter, quant=quant, **c)
    w, ws = R.make_weights(_gen(inter + c["k"]), rows.E, 2 * inter, c["k"], quant, "cuda")
    h = _filled((rows.rows, inter), torch.uint8)
    hs = _scales(rows.rows, inter, quant)
    M.moe_expert_gemm_swiglu(rows.cfg, c["T"], inter, rows.a, rows.s, w, ws, rows.handle, h, hs)
    torch.cuda.synchronize()
    _untouched(h[~rows.used], "rows without a pair")
    _untouched(hs[~rows.used], "scales without a pair")
    for e, (o, m) in enumerate(zip(rows.off, rows.count)):
        if m == 0:
            continue
        a = R.dequantize(rows.a[o:o + m], rows.s[o:o + m], quant)[:300]
        wv = R.weight_values(w[e:e + 1], ws[e:e + 1], quant)[0]
        y, bound = R.product(a, wv)
        g, u, dg, du = y[:, :inter], y[:, inter:], bound[:, :inter], bound[:, inter:]
        want = R.silu(g) * u
        # |silu'| <= 1.1; the function itself in fp32 (an exponential of argument g: |g| ulps)
        lim = 1.1 * dg * (u.abs() + du) + R.silu(g).abs() * du + want.abs() * (8 + g.abs()) * 2.0 ** -24
        R.assert_rows(h[o:o + m][:300], hs[o:o + m][:300], want, lim, quant, f"expert {e}")
        if quant == M.QUANT_FP8_UE8M0 and (inter // 128) % 4:
            assert not bool(hs[o:o + m].view(torch.uint8)[:, inter // 128:].any())
        if quant == M.QUANT_FP8_F32:
            ref = R.block_scale((R.silu(g) * u).abs().unflatten(-1, (-1, 128)).amax(-1), quant)
            # stored fp32 scales: 1e-5 of them, as a whole
            assert float((hs[o:o + m][:300].to(D) - ref).norm() / ref.norm()) <= 1e-5


def test_products_read_weights_past_4_gib():
    """The last expert's weights lie beyond 32-bit byte offsets."""
    E, n, k, T = 33, 16384, 8192, 3
    _say(f"weights of {E * n * k / 2**30:.1f} GiB, rows of the last expert only")
    quant = M.QUANT_FP8_UE8M0
    for tokens in (T, 40):  # 16-row and 128-row tiles (by the average per expert: one expert for the latter)
        w = torch.zeros(E, n, k, dtype=torch.uint8, device="cuda")
        ws = torch.full((E, n // 128, k // 512), 0x77777777, dtype=torch.int32, device="cuda")
        last, _ = R.make_weights(_gen(4), 1, n, k, quant, "cuda")
        w[E - 1] = last[0]
        cfg = _cfg(tokens, k, E, 1, quant)
        idx = torch.full((tokens, 1), E - 1, dtype=torch.int32, device="cuda")
        handle = M.Handle(cfg)
        lw = torch.empty(M.moe_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
        M.moe_dispatch_layout(cfg, tokens, idx, handle, lw)
        a, s = R.quantize(torch.randn(tokens, k, generator=_gen(8), device="cuda"), quant)
        y = torch.empty(tokens, n, dtype=torch.bfloat16, device="cuda")
        M.moe_expert_gemm(cfg, tokens, n, k, a, s, w, ws, handle, y)
        torch.cuda.synchronize()
        wv = R.weight_values(w[E - 1:], ws[E - 1:], quant)[0]
        want = R.dequantize(a, s, quant) @ wv.T
        assert float((y.to(D) - want).norm() / want.norm()) <= 2.0 ** -8 + 2.0 ** -15


@pytest.mark.parametrize("quant", FORMATS)
def test_products_do_not_depend_on_when_loads_arrive(quant):
    """Blocks that go from tile to tile, each a few rows of another expert, with weights and
    rows from memory (a buffer larger than the caches is written between): every run gives
    the same bits, and the sums of the formulas."""
    _say(f"products of many small tiles, caches cold, quant {quant}")
    case = dict(T=96, E=64, K=6, k=1024)
    rows = Rows(5, quant=quant, **case)
    n, inter = 4096, 2048
    w, ws = R.make_weights(_gen(6), 64, n, 1024, quant, "cuda")
    cold = torch.empty(1 << 29, dtype=torch.uint8, device="cuda")
    first = None
    for i in range(8):
        y = _filled((rows.rows, n), torch.bfloat16)
        h = _filled((rows.rows, inter), torch.uint8)
        hs = _scales(rows.rows, inter, quant)
        cold.fill_(i)
        M.moe_expert_gemm(rows.cfg, 96, n, 1024, rows.a, rows.s, w, ws, rows.handle, y)
        cold.fill_(i)
        M.moe_expert_gemm_swiglu(rows.cfg, 96, inter, rows.a, rows.s, w, ws, rows.handle, h, hs)
        torch.cuda.synchronize()
        got = [y[rows.used].view(torch.int16), h[rows.used], hs[rows.used].view(torch.int32)]
        if first is None:
            first = got
        for a, b in zip(first, got):
            assert torch.equal(a, b), i
    for e in (0, 21, 42, 63):
        o, m = rows.off[e], rows.count[e]
        a = R.dequantize(rows.a[o:o + m], rows.s[o:o + m], quant)
        want, bound = R.product(a, R.weight_values(w[e:e + 1], ws[e:e + 1], quant)[0])
        R.assert_bf16(y[o:o + m], want, bound, f"expert {e}")


def test_products_without_rows():
    _say("no token, and tokens that route nowhere")
    cfg = _cfg(8, 256, 4, 2, M.QUANT_FP8_F32, align=128)
    handle = M.Handle(cfg)
    lw = torch.empty(M.moe_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    idx = torch.full((8, 2), -1, dtype=torch.int32, device="cuda")
    rows = M.moe_rows_capacity(cfg)
    a, s = _filled((rows, 256), torch.uint8), _scales(rows, 256, M.QUANT_FP8_F32)
    w, ws = R.make_weights(_gen(1), 4, 256, 256, M.QUANT_FP8_F32, "cuda")
    y = _filled((rows, 256), torch.bfloat16)
    for T in (8, 0):
        M.moe_dispatch_layout(cfg, T, idx, handle, lw)
        M.moe_expert_gemm(cfg, T, 256, 256, a, s, w, ws, handle, y)
        torch.cuda.synchronize()
        _untouched(y, f"T={T}")


# ---- few-token layer ----------------------------------------------------------------------


def _layer_reference(idx, tw, x, w13, s13, w2, s2, quant, inter):
    """out and a bound: bf16 h (half a step each), fp32 sums."""
    T, H = x.shape
    out = torch.zeros(T, H, dtype=D, device="cuda")
    bound = torch.zeros_like(out)
    for e in range(w13.shape[0]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if t.numel() == 0:
            continue
        a = R.weight_values(w13[e:e + 1], None if s13 is None else s13[e:e + 1], quant)[0]
        b = R.weight_values(w2[e:e + 1], None if s2 is None else s2[e:e + 1], quant)[0]
        y, d = R.product(x[t].to(D), a, eight_bit=False)
        g, u, dg, du = y[:, :inter], y[:, inter:], d[:, :inter], d[:, inter:]
        h = R.silu(g) * u
        dh = (1.1 * dg * (u.abs() + du) + R.silu(g).abs() * du + h.abs() * (8 + g.abs()) * 2.0 ** -24)
        dh = dh + (h.abs() + dh) * 2.0 ** -8
        wt = tw[t, j].to(D).unsqueeze(-1)
        z, dz = R.product(h, b, eight_bit=False)
        out.index_add_(0, t, z * wt)
        bound.index_add_(0, t, (dz + dh @ b.abs().T) * wt.abs())
    return out, bound + out.abs() * 64 * 2.0 ** -24


LAYERS = [
    dict(T=1, E=8, K=1, H=128, inter=128),
    dict(T=1, E=16, K=8, H=1024, inter=640),
    dict(T=2, E=3, K=2, H=512, inter=256),
    dict(T=5, E=40, K=8, H=2048, inter=768),
    dict(T=16, E=4, K=2, H=384, inter=128, holes=0.4),
    dict(T=17, E=300, K=4, H=256, inter=256),           # more experts than pairs
    dict(T=33, E=8, K=3, H=640, inter=384, holes=0.2),
    dict(T=64, E=6, K=2, H=256, inter=128),             # more than 16 tokens of one expert
    dict(T=64, E=2, K=1, H=128, inter=256),
    dict(T=3, E=4, K=2, H=8192, inter=128),             # wide outputs
    dict(T=40, E=64, K=32, H=128, inter=128),           # the largest top-k
    dict(T=64, E=2048, K=32, H=128, inter=128),         # as many pairs as experts, most used
]


@pytest.mark.parametrize("quant", [M.QUANT_NONE] + FORMATS)
@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "T{T}_E{E}_K{K}_H{H}_i{inter}".format(**c))
def test_layer_fused(case, quant):
    _say(f"layer_fused {case} quant={quant}")
    c = dict(case)
    T, E, K, H, inter = c["T"], c["E"], c["K"], c["H"], c["inter"]
    g = _gen(T + E + H)
    idx = torch.topk(torch.rand(T, E, generator=g, device="cuda"), K, 1).indices.to(torch.int32)
    if c.get("holes"):
        idx[torch.rand(T, K, generator=g, device="cuda") < c["holes"]] = -1
        idx[0, 0] = E
        idx[T - 1] = -1                                  # a token without pairs
    if T > 2 and K > 1:
        idx[1, 1] = idx[1, 0]                            # the same expert twice
    tw = torch.rand(T, K, generator=g, device="cuda")
    tw[(idx < 0) | (idx >= E)] = float("nan")            # weights of pairs that do not count
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w13, s13 = R.make_weights(g, E, 2 * inter, H, quant, "cuda")
    w2, s2 = R.make_weights(g, E, H, inter, quant, "cuda")
    cfg = _cfg(T, H, E, K, quant)
    need = M.moe_layer_workspace_bytes(cfg, inter)
    ws = _filled((need + 256,), torch.uint8)
    out = _filled((T + 1, H), torch.bfloat16)
    M.moe_layer_fused(cfg, T, inter, idx, tw, x, w13, s13, w2, s2, ws[:need], out)
    torch.cuda.synchronize()
    _untouched(ws[need:], "behind the workspace")
    _untouched(out[T:], "row behind the last token")
    want, bound = _layer_reference(idx, tw, x, w13, s13, w2, s2, quant, inter)
    R.assert_bf16(out[:T], want, bound, "out")
    # both roundings of half a step, as a whole
    assert float((out[:T].to(D) - want).norm()) <= 2.0 ** -7 * float(want.norm()) + 1e-30
    if c.get("holes"):
        assert not bool(out[T - 1].view(torch.int16).any())
    again = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    M.moe_layer_fused(cfg, T, inter, idx, tw, x, w13, s13, w2, s2, ws[:need], again)
    torch.cuda.synchronize()
    assert torch.equal(again.view(torch.int16), out[:T].view(torch.int16))


# ---- together ----------------------------------------------------------------------------------


class Chain:
    """norm -> dispatch -> gate/up -> down -> combine, and the few-token layer on the same tokens."""

    def __init__(self, seed, T=48, H=512, E=16, K=4, inter=256, quant=M.QUANT_FP8_UE8M0, layout=M.LAYOUT_CONTIGUOUS,
                 align=16, capacity=32):
        g = _gen(seed)
        self.T, self.H, self.inter, self.quant = T, H, inter, quant
        self.cfg = _cfg(T, H, E, K, quant, layout, align, capacity)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.x, self.res = rn(T, H).bfloat16(), rn(T, H).bfloat16()
        self.nw = (1 + 0.1 * rn(H)).bfloat16()
        self.idx = torch.topk(torch.rand(T, E, generator=g, device="cuda"), K, 1).indices.to(torch.int32)
        self.tw = torch.softmax(rn(T, K), -1)
        self.w13, self.s13 = R.make_weights(g, E, 2 * inter, H, quant, "cuda")
        self.w2, self.s2 = R.make_weights(g, E, H, inter, quant, "cuda")
        self.bufs = M.DispatchBuffers(self.cfg)
        e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.normed, self.res_out, self.out, self.out_few = (e(T, H) for _ in range(4))
        self.q, self.qs = torch.empty(T, H, dtype=torch.uint8, device="cuda"), _scales(T, H, quant)
        rows = self.bufs.rows
        self.h, self.hs = torch.empty(rows, inter, dtype=torch.uint8, device="cuda"), _scales(rows, inter, quant)
        self.y = e(rows, H)
        self.ws = torch.empty(M.moe_layer_workspace_bytes(self.cfg, inter), dtype=torch.uint8, device="cuda")
        # a shared expert: the same kernels without a handle
        self.shared_cfg = _cfg(T, H, quant=quant)
        self.sw13, self.ss13 = R.make_weights(g, 1, 2 * inter, H, quant, "cuda")
        self.sw2, self.ss2 = R.make_weights(g, 1, H, inter, quant, "cuda")
        self.sh, self.shs, self.sy = torch.empty(T, inter, dtype=torch.uint8, device="cuda"), _scales(T, inter, quant), e(T, H)

    def run(self):
        c, T, b = self.cfg, self.T, self.bufs
        M.moe_rmsnorm(c, T, self.x, self.res, self.nw, 1e-6, self.res_out, self.normed, self.q, self.qs)
        M.moe_dispatch_fused(c, T, self.idx, self.normed, None, b.handle, b.workspace, b.out_x, b.out_scale)
        M.moe_expert_gemm_swiglu(c, T, self.inter, b.out_x, b.out_scale, self.w13, self.s13, b.handle, self.h, self.hs)
        M.moe_expert_gemm(c, T, self.H, self.inter, self.h, self.hs, self.w2, self.s2, b.handle, self.y)
        M.moe_combine(c, T, self.y, self.tw, b.handle, self.out)
        M.moe_expert_gemm_swiglu(self.shared_cfg, T, self.inter, self.q, self.qs, self.sw13, self.ss13, None, self.sh,
                                 self.shs)
        M.moe_expert_gemm(self.shared_cfg, T, self.H, self.inter, self.sh, self.shs, self.sw2, self.ss2, None, self.sy)
        M.moe_layer_fused(c, T, self.inter, self.idx, self.tw, self.normed, self.w13, self.s13, self.w2, self.s2,
                          self.ws, self.out_few)

    def outputs(self):
        return {k: getattr(self, k).clone() for k in ("res_out", "normed", "q", "qs", "out", "sy", "out_few")}


@pytest.mark.parametrize("quant", FORMATS)
@pytest.mark.parametrize("layout", [M.LAYOUT_CONTIGUOUS, M.LAYOUT_MASKED])
def test_a_layer_end_to_end(quant, layout):
    _say(f"norm, dispatch, experts, combine, shared expert, few-token layer: quant={quant} layout={layout}")
    c = Chain(21, quant=quant, layout=layout)
    c.run()
    torch.cuda.synchronize()
    want, bound = _layer_reference(c.idx, c.tw, c.normed, c.w13, c.s13, c.w2, c.s2, quant, c.inter)
    R.assert_bf16(c.out_few, want, bound, "few-token layer")
    # the dispatched path quantizes x and h to E4M3: each value is off by at most 2^-4 of itself (MXFP8
    # saturates its largest by up to 1/8), an error of independent sign in every term of a sum
    few = float((c.out.to(D) - want).norm() / want.norm())
    assert few <= 0.125 * 2 ** 0.5, few
    # the shared expert against the reference on the same 8-bit rows
    a = R.dequantize(c.q, c.qs, quant)
    y = a @ R.weight_values(c.sw13, c.ss13, quant)[0].T
    h = R.silu(y[:, :c.inter]) * y[:, c.inter:]
    own = R.dequantize(c.sh, c.shs, quant)
    assert float((own - h).norm() / h.norm()) <= 2.0 ** -4
    down = own @ R.weight_values(c.sw2, c.ss2, quant)[0].T
    assert float((c.sy.to(D) - down).norm() / down.norm()) <= 2.0 ** -8 + 2.0 ** -15


def test_captured_and_replayed():
    _say("a layer captured into a graph, replayed with eager work between")
    c = Chain(31, quant=M.QUANT_FP8_F32)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    g = _gen(77)
    for _ in range(4):
        c.x.copy_(torch.randn(c.T, c.H, generator=g, device="cuda").bfloat16())
        c.idx.copy_(torch.topk(torch.rand(c.T, 16, generator=g, device="cuda"), 4, 1).indices.to(torch.int32))
        c.run()
        torch.cuda.synchronize()
        want = c.outputs()
        for t in (c.out, c.out_few, c.sy, c.normed, c.q, c.res_out):
            t.view(torch.uint8).fill_(SENT)
        graph.replay()
        torch.cuda.synchronize()
        for k, v in c.outputs().items():
            assert torch.equal(v.view(torch.uint8), want[k].view(torch.uint8)), k


def test_two_streams_with_their_own_buffers():
    _say("two layers on two streams at once")
    chains = [Chain(41, quant=M.QUANT_MXFP8), Chain(42, T=9, H=1024, quant=M.QUANT_FP8_F32)]
    want = []
    for c in chains:
        c.run()
        torch.cuda.synchronize()
        want.append(c.outputs())
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(3):
        for c, s in zip(chains, streams):
            with torch.cuda.stream(s):
                c.run()
    torch.cuda.synchronize()
    for c, w in zip(chains, want):
        for k, v in c.outputs().items():
            assert torch.equal(v.view(torch.uint8), w[k].view(torch.uint8)), k


def test_binding_refusals():
    _say("what the binding refuses before the library is called")
    c = Chain(51)
    T, H = c.T, c.H
    args = (c.cfg, T, H, c.inter, c.h, c.hs, c.w2, c.s2, c.bufs.handle, c.y)

    def put(i, v):
        return args[:i] + (v,) + args[i + 1:]
    with pytest.raises(ValueError, match="elements <"):
        M.moe_expert_gemm(*put(9, c.y[:-1]))
    with pytest.raises(ValueError, match="contiguous"):
        M.moe_expert_gemm(*put(6, c.w2.transpose(1, 2)))
    with pytest.raises(ValueError, match="byte elements"):
        M.moe_expert_gemm(*put(4, c.h.view(torch.int16)))
    with pytest.raises(ValueError, match="device"):
        M.moe_expert_gemm(*put(4, c.h.cpu()))
    with pytest.raises(ValueError, match="elements <"):
        M.moe_expert_gemm(*put(7, c.s2[:, :-1].contiguous()))
    with pytest.raises(M.MoeError) as e:
        M.moe_expert_gemm(_cfg(T, H, 16, 4, M.QUANT_NONE), *args[1:])
    assert e.value.code == M.MOE_ERR_UNSUPPORTED
    with pytest.raises(ValueError, match="without FP8"):
        M.moe_rmsnorm(_cfg(T, H, quant=M.QUANT_NONE), T, c.x, None, c.nw, 1e-6, None, c.normed, c.q, c.qs)
    with pytest.raises(M.MoeError) as e:
        M.moe_layer_fused(c.cfg, T, c.inter, c.idx, c.tw, c.x, c.w13, c.s13, c.w2, c.s2, c.ws[:64], c.out_few)
    assert e.value.code == M.MOE_ERR_CAPACITY
