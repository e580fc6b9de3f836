"""The bf16 expert layer's operators where every large array passes 2^32 bytes.

Two experts with 16,601 rows each; rows on both sides of 2^31 and 2^32 bytes of
each array and rows picked at random are compared with the 64-bit reference.
Outputs lie in sentinel-filled buffers: a row that was written elsewhere shows
as one that was not written, and the rows between the experts and behind the
last are compared byte for byte.  Channels are 128 * 513 and twice that.
"""
import pytest
import torch

import combine_topk_idx_amd as M
import strict_reference as S
import train_reference as R
from test_gpu_train import BF16, D, FP8, MX, UE8M0, Rows, _filled, _format_buffers, _gen, _gpu, _say, _untouched, _weights  # noqa: F401

pytestmark = pytest.mark.gpu
T, N = 16601, 128 * 513


def _rows(H):
    rows = Rows(T, H, 2, 2, "contiguous", align=128, seed=3)
    assert [hi - lo for lo, hi in rows.spans] == [T, T]
    return rows


def _picked(rows, *row_bytes):
    """(expert, rows) to compare: the experts' first and last ones, those at 2^31 and 2^32 bytes of arrays with
    row_bytes, and 40 others."""
    at = {r for lo, hi in rows.spans for r in (lo, lo + 255, hi - 1)}
    for b in row_bytes:
        for limit in (1 << 31, 1 << 32):
            at |= {limit // b - 1, limit // b, limit // b + 1}
    at |= set(torch.randint(rows.n, (40,), generator=torch.Generator().manual_seed(1)).tolist())
    for e, (lo, hi) in enumerate(rows.spans):
        yield e, torch.tensor(sorted(r for r in at if lo <= r < hi), device="cuda")


def _unused(rows, *outputs):
    unused = torch.nonzero(~rows.live).squeeze(1)
    for t in outputs:
        _untouched(t[unused], "rows without a pair")


def _compare_saved(q, s, quant, at, v, b):
    if quant == BF16:
        S.assert_bf16(q[at], v, b, "saved")
    else:
        R.assert_rows(q[at], s[at], v, b, quant, "saved")


@pytest.mark.parametrize("save", [BF16, FP8, UE8M0, MX])
def test_gated(save):
    _say(f"gated past 4 GiB save={save}")
    k, rows = 72, _rows(72)
    g = _gen(save)
    a, w = rows.input(g, k), _weights(g, 2, 2 * N, k)
    h = _filled((rows.n + 2, N), torch.bfloat16)
    q, s = _format_buffers(rows.n + 2, 2 * N, save)
    assert h.numel() * 2 > 1 << 32 and q.numel() * q.element_size() > 1 << 32
    M.moe_ffn_gated(rows.cfg, T, N, M.ACT_SILU, a, w, rows.handle, h, q, s, save)
    torch.cuda.synchronize()
    for e, at in _picked(rows, 2 * N, 2 * N * q.element_size()):
        p, b = R.product(a[at].to(D), w[e].to(D))
        S.assert_bf16(h[at], *R.gated(p, b, R.SILU), "h")
        _compare_saved(q, s, save, at, p, b)
    _unused(rows, h, q, *([] if s is None else [s]))


@pytest.mark.parametrize("save", [BF16, UE8M0])
def test_linear(save):
    _say(f"linear past 4 GiB save={save}")
    k, n, rows = 72, 2 * N, _rows(8)
    g = _gen(10 + save)
    a, w = rows.input(g, k), _weights(g, 2, n, k)
    bias = torch.randn(2, n, generator=g, device="cuda").bfloat16()
    res = torch.randn(rows.n + 2, n, generator=g, device="cuda", dtype=torch.bfloat16)
    y = _filled((rows.n + 2, n), torch.bfloat16)
    q, s = _format_buffers(rows.n + 2, n, save)
    assert q.numel() * q.element_size() > 1 << 32
    M.moe_expert_linear(rows.cfg, T, n, k, M.ACT_GELU, a, w, bias, res, rows.handle, y, q, s, save)
    torch.cuda.synchronize()
    for e, at in _picked(rows, 2 * n, n * q.element_size()):
        p, b = R.product(a[at].to(D), w[e].to(D))
        p = p + bias[e].to(D)
        b = b + p.abs() * 2.0 ** -23
        _compare_saved(q, s, save, at, p, b)
        v = R.act(p, R.GELU)[0]
        b = R.act_bound(p, v, b, R.GELU)
        v = v + res[at].to(D)
        S.assert_bf16(y[at], v, b + v.abs() * 2.0 ** -23, "y")
    _unused(rows, y, q, *([] if s is None else [s]))


@pytest.mark.parametrize("quant,gated", [(BF16, False), (BF16, True), (FP8, True), (UE8M0, False), (MX, True)])
def test_activation_backward(quant, gated):
    _say(f"activation backward past 4 GiB quant={quant} gated={gated}")
    # 8-bit rows pass 2^32 bytes with 2 N channels
    n, m, rows = (N, 2 * N, _rows(8)) if gated else (2 * N, 2 * N, _rows(8))
    g = _gen(20 + quant)
    dy = torch.randn(rows.n + 2, n, generator=g, device="cuda", dtype=torch.bfloat16)
    if quant == BF16:
        q, s = torch.randn(rows.n + 2, m, generator=g, device="cuda", dtype=torch.bfloat16), None
    else:  # any byte but the two NaNs is a value, any scale in (0.5, 2)
        q = torch.randint(0, 0x7F, (rows.n + 2, m), generator=g, device="cuda", dtype=torch.uint8)
        q |= torch.randint(0, 2, (rows.n + 2, m), generator=g, device="cuda", dtype=torch.uint8) << 7
        s = _format_buffers(rows.n + 2, m, quant)[1]
        if quant == FP8:
            s.copy_((torch.rand(s.shape, generator=g, device="cuda") + 0.5) / 64)
        else:
            s.view(torch.uint8).copy_(torch.randint(120, 123, s.view(torch.uint8).shape, generator=g, device="cuda"))
    ds, y = _filled((rows.n + 2, m), torch.bfloat16), _filled((rows.n + 2, n), torch.bfloat16)
    assert q.numel() * q.element_size() > 1 << 32 and y.numel() * 2 > 1 << 32
    M.moe_activation_backward(rows.cfg, T, n, M.ACT_SILU, gated, dy, q, s, quant, rows.handle, ds, y)
    torch.cuda.synchronize()
    picked = list(_picked(rows, 2 * n, 2 * m, m * q.element_size()))
    for _, at in picked:
        saved = q[at].to(D) if quant == BF16 else R.dequantize(q[at], s[at], quant)
        (v, b), (f, bf) = R.act_grads(dy[at].to(D), saved, R.SILU, gated)
        S.assert_bf16(ds[at], v, b, "dsaved")
        S.assert_bf16(y[at], f, bf, "y")
    _unused(rows, ds, y)
    if quant != BF16:
        return
    M.moe_activation_backward(rows.cfg, T, n, M.ACT_SILU, gated, dy, q, s, quant, rows.handle, q, dy)  # into its own arrays
    torch.cuda.synchronize()
    for _, at in picked:
        assert torch.equal(q[at], ds[at]) and torch.equal(dy[at], y[at])


def test_grad_input():
    _say("grad input past 4 GiB")
    n, k, rows = 72, N, _rows(8)
    g = _gen(30)
    dy, w = rows.input(g, n, 0.02), _weights(g, 2, n, k)
    da = _filled((rows.n + 2, k), torch.bfloat16)
    M.moe_expert_grad_input(rows.cfg, T, n, k, dy, w, rows.handle, da)
    wide = torch.randn(rows.n + 2, k, generator=g, device="cuda", dtype=torch.bfloat16)  # and rows of the sum's own
    wide[~rows.live] = float("nan")
    small, back = _filled((rows.n + 2, n), torch.bfloat16), _weights(g, 2, k, n)
    M.moe_expert_grad_input(rows.cfg, T, k, n, wide, back, rows.handle, small)
    torch.cuda.synchronize()
    for e, at in _picked(rows, 2 * k):
        S.assert_bf16(da[at], *R.product(dy[at].to(D), w[e].to(D).T), "da")
        S.assert_bf16(small[at], *R.product(wide[at].to(D), back[e].to(D).T), "da of wide rows")
    _unused(rows, da, small)


@pytest.mark.parametrize("quant", [BF16, FP8, UE8M0, MX])
def test_grad_weight(quant):
    """Rows that are zeros but for those picked: every one of them counts once."""
    _say(f"grad weight past 4 GiB quant={quant}")
    n, k, rows = 8, 2 * N, _rows(8)
    g = _gen(40 + quant)
    dy = rows.input(g, n)
    picked = [at for _, at in _picked(rows, 2 * k, k)]
    at = torch.cat(picked)
    a, s = torch.zeros(rows.n + 2, k, dtype=torch.bfloat16 if quant == BF16 else torch.uint8, device="cuda"), None
    x = torch.randn(at.numel(), k, generator=g, device="cuda").bfloat16()
    if quant == BF16:
        a[at] = x
    else:
        q, sq = R.quantize(x.float(), quant)
        s = torch.zeros(rows.n + 2, sq.shape[1], dtype=sq.dtype, device="cuda")
        a[at], s[at] = q, sq
    assert a.numel() * a.element_size() > 1 << 32
    dw, db = _filled((3, n, k), torch.float32), _filled((3, n), torch.float32)
    size = M.moe_grad_weight_workspace_bytes(rows.cfg, T, n, k)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    M.moe_expert_grad_weight(rows.cfg, T, n, k, dy, a, s, quant, rows.handle, dw, db, False, ws)
    torch.cuda.synchronize()
    for e, r in enumerate(picked):
        d = dy[r].to(D)
        v = a[r].to(D) if quant == BF16 else R.dequantize(a[r], s[r], quant).float().bfloat16().to(D)
        want, bound = R.product(d.T, v.T)  # the other rows add zeros, which are exact
        R.assert_near(dw[e], want, bound, f"dw[{e}]")
        lo, hi = rows.spans[e]
        all_ = dy[lo:hi].to(D)
        R.assert_near(db[e], all_.sum(0), (T + 8) * 2.0 ** -23 * all_.abs().sum(0), f"dbias[{e}]")
    _untouched(dw[2], "dw behind the last expert")


def test_combine_backward():
    _say("combine backward past 4 GiB")
    H, rows = N, _rows(N)
    g = _gen(50)
    dout = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    y = torch.randn(rows.n + 2, H, generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(T, 2, generator=g, device="cuda") + 0.1
    dy, dw = _filled((rows.n + 2, H), torch.bfloat16), _filled((T + 1, 2), torch.float32)
    M.moe_combine_backward(rows.cfg, T, dout, y, w, rows.handle, dy, dw)
    torch.cuda.synchronize()
    pair = rows.handle.row_to_pair
    for _, at in _picked(rows, 2 * H):
        p = pair[at].long()
        d = dout[p // 2].to(D)
        v = d * w.view(-1)[p].to(D).unsqueeze(1)
        S.assert_bf16(dy[at], v, v.abs() * 2.0 ** -23, "dy")
        terms = d * y[at].to(D)
        R.assert_near(dw.view(-1)[p], terms.sum(1), (H + 8) * 2.0 ** -23 * terms.abs().sum(1), "dtopk_w")
    _unused(rows, dy)
    _untouched(dw[T], "dtopk_w")
