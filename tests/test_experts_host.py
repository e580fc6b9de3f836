"""Host-side tests of the expert-layer operators (no GPU needed): exported
symbols, size queries, every refusal of the C ABI (decided before anything is
enqueued; pointers are fake aligned addresses), the binding's own checks, and
the 64-bit reference against the CPU oracle's quantizer."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import combine_topk_idx_amd as M
import expert_reference as R
import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_experts.h")
FAKE = 0x7F0000000000  # never dereferenced
NAMES = ["moe_expert_gemm", "moe_expert_gemm_swiglu", "moe_layer_fused", "moe_layer_workspace_bytes", "moe_rmsnorm"]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.LIB_PATH):
        pytest.fail("libmoe_dispatch.so is not built (python -m combine_topk_idx_amd.build)")
    return M.library()


def _cfg(**kw):
    base = dict(max_tokens=64, hidden=256, num_experts=8, num_topk=2, num_ranks=2,
                layout=M.LAYOUT_CONTIGUOUS, align=1, capacity=1, quant=M.QUANT_FP8_F32, num_cus=0)
    base.update(kw)
    return M.MoeConfig(**base)


def _handle(**override):
    vals = {n: FAKE + 0x1000 * i for i, (n, _) in enumerate(M.MoeHandle._fields_)}
    vals.update(override)
    return M.MoeHandle(**vals)


def test_header_declares_and_library_exports(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(moe_[a-z_]+)\s*\(", src))) == NAMES
    out = subprocess.run(["nm", "-D", "--defined-only", M.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r"\bT (moe_[a-z_]+)\b", out))
    assert not [n for n in NAMES if n not in exported]


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "moe_experts.h"\nint main(void) { return MOE_LAYER_MAX_TOKENS != 64; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    "-fsyntax-only", str(src)], check=True)


# ---- moe_rmsnorm ----------------------------------------------------------------

NORM_OK = dict(x=FAKE, residual=FAKE, weight=FAKE, eps=1e-6, residual_out=FAKE, out=FAKE, out_q=FAKE, out_scale=FAKE)


def _norm(lib, cfg, T, **kw):
    a = dict(NORM_OK, **kw)
    return lib.moe_rmsnorm(ctypes.byref(cfg) if cfg is not None else None, T, a["x"], a["residual"], a["weight"],
                           a["eps"], a["residual_out"], a["out"], a["out_q"], a["out_scale"], None)


@pytest.mark.parametrize("cfg,T,kw,code", [
    (None, 1, {}, M.MOE_ERR_INVALID_ARG),
    (dict(num_topk=0), 1, {}, M.MOE_ERR_INVALID_ARG),
    (dict(), -1, {}, M.MOE_ERR_INVALID_ARG),
    (dict(), 65, {}, M.MOE_ERR_CAPACITY),
    (dict(hidden=32768 + 128), 1, {}, M.MOE_ERR_UNSUPPORTED),
    (dict(), 1, dict(eps=0.0), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(eps=-1e-6), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(eps=float("nan")), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(eps=float("inf")), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(residual=None), M.MOE_ERR_INVALID_ARG),            # residual_out without residual
    (dict(), 1, dict(residual_out=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(out_q=None), M.MOE_ERR_INVALID_ARG),               # scales without rows
    (dict(), 1, dict(out_scale=None), M.MOE_ERR_INVALID_ARG),
    (dict(quant=M.QUANT_NONE), 1, {}, M.MOE_ERR_INVALID_ARG),           # 8-bit rows without a format
    (dict(), 1, dict(out=None, out_q=None, out_scale=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(x=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(weight=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(x=FAKE + 8), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(residual=FAKE + 2), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(residual_out=FAKE + 2), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(out=FAKE + 2), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(out_q=FAKE + 8), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(out_scale=FAKE + 2), M.MOE_ERR_INVALID_ARG),
    (dict(), 0, {}, M.MOE_OK),
    (dict(), 0, dict(x=None, weight=None), M.MOE_OK),
])
def test_rmsnorm_refusals(lib, cfg, T, kw, code):
    assert _norm(lib, None if cfg is None else _cfg(**cfg), T, **kw) == code


# ---- products --------------------------------------------------------------------

GEMM_OK = dict(n=256, k=256, a=FAKE, a_scale=FAKE, w=FAKE, w_scale=FAKE, handle=True, y=FAKE)


def _gemm(lib, cfg, T, **kw):
    a = dict(GEMM_OK, **kw)
    h = a["handle"]
    hp = None if h is None else ctypes.byref(_handle(**(h if isinstance(h, dict) else {})))
    return lib.moe_expert_gemm(ctypes.byref(cfg) if cfg is not None else None, T, a["n"], a["k"], a["a"], a["a_scale"],
                               a["w"], a["w_scale"], hp, a["y"], None)


@pytest.mark.parametrize("cfg,T,kw,code", [
    (None, 1, {}, M.MOE_ERR_INVALID_ARG),
    (dict(num_ranks=3), 1, {}, M.MOE_ERR_INVALID_ARG),
    (dict(quant=M.QUANT_NONE), 1, {}, M.MOE_ERR_UNSUPPORTED),
    (dict(), -1, {}, M.MOE_ERR_INVALID_ARG),
    (dict(), 65, {}, M.MOE_ERR_CAPACITY),
    (dict(), 1, dict(n=0), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(n=-8), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(n=12), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(k=0), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(k=192), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(k=(1 << 22) + 128), M.MOE_ERR_UNSUPPORTED),
    (dict(), 1, dict(n=1 << 20, k=1 << 17), M.MOE_ERR_UNSUPPORTED),     # an expert's scales past 2 GiB
    (dict(), 1, dict(handle=dict(recv_count=None)), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(handle=dict(expert_offset=FAKE + 2)), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(handle=None), M.MOE_ERR_INVALID_ARG),              # dense needs one expert
    (dict(), 1, dict(a=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(a=FAKE + 8), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(a_scale=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(a_scale=FAKE + 2), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(w=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(w=FAKE + 4), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(w_scale=None), M.MOE_ERR_INVALID_ARG),
    (dict(quant=M.QUANT_MXFP8), 1, dict(w_scale=FAKE + 1), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(y=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(y=FAKE + 8), M.MOE_ERR_INVALID_ARG),
    (dict(), 0, {}, M.MOE_OK),
    (dict(), 0, dict(a=None, a_scale=None, w=None, w_scale=None, y=None), M.MOE_OK),
    (dict(num_experts=1, num_topk=1, num_ranks=1), 0, dict(handle=None), M.MOE_OK),
])
def test_gemm_refusals(lib, cfg, T, kw, code):
    assert _gemm(lib, None if cfg is None else _cfg(**cfg), T, **kw) == code


@pytest.mark.parametrize("cfg,T,kw,code", [
    (None, 1, {}, M.MOE_ERR_INVALID_ARG),
    (dict(quant=M.QUANT_NONE), 1, {}, M.MOE_ERR_UNSUPPORTED),
    (dict(), 1, dict(inter=0), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(inter=64), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(inter=200), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(inter=(1 << 30) + 128), M.MOE_ERR_INVALID_ARG),
    (dict(), 65, {}, M.MOE_ERR_CAPACITY),
    (dict(), 1, dict(h=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(h=FAKE + 8), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(h_scale=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(h_scale=FAKE + 2), M.MOE_ERR_INVALID_ARG),
    (dict(), 0, {}, M.MOE_OK),
])
def test_swiglu_refusals(lib, cfg, T, kw, code):
    a = dict(inter=256, h=FAKE, h_scale=FAKE)
    a.update(kw)
    c = None if cfg is None else ctypes.byref(_cfg(**cfg))
    assert lib.moe_expert_gemm_swiglu(c, T, a["inter"], FAKE, FAKE, FAKE, FAKE, ctypes.byref(_handle()), a["h"],
                                      a["h_scale"], None) == code


def test_output_channels_past_the_limit(lib):
    """256 rows of more than 2^22 output channels pass the products' 32-bit offsets."""
    assert _gemm(lib, _cfg(), 0, n=1 << 22, k=128) == M.MOE_OK
    assert _gemm(lib, _cfg(), 1, n=(1 << 22) + 8, k=128) == M.MOE_ERR_UNSUPPORTED


# ---- few-token layer ----------------------------------------------------------------

LAYER_OK = dict(inter=256, topk_idx=FAKE, topk_w=FAKE, x=FAKE, w13=FAKE, w13_scale=FAKE, w2=FAKE, w2_scale=FAKE,
                ws=FAKE, ws_bytes=1 << 30, out=FAKE)


@pytest.mark.parametrize("cfg,T,kw,code", [
    (None, 1, {}, M.MOE_ERR_INVALID_ARG),
    (dict(num_experts=0), 1, {}, M.MOE_ERR_INVALID_ARG),
    (dict(quant=M.QUANT_NONE, hidden=200), 1, dict(w13_scale=None, w2_scale=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(inter=0), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(inter=192), M.MOE_ERR_INVALID_ARG),
    (dict(), -1, {}, M.MOE_ERR_INVALID_ARG),
    (dict(), 65, {}, M.MOE_ERR_CAPACITY),
    (dict(max_tokens=100), 65, {}, M.MOE_ERR_UNSUPPORTED),
    (dict(), 1, dict(topk_idx=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(topk_w=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(topk_w=FAKE + 2), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(x=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(x=FAKE + 8), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(w13=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(w2=FAKE + 8), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(w13_scale=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(w2_scale=None), M.MOE_ERR_INVALID_ARG),
    (dict(quant=M.QUANT_NONE), 1, {}, M.MOE_ERR_INVALID_ARG),           # scales with bf16 weights
    (dict(), 1, dict(ws=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(ws=FAKE + 8), M.MOE_ERR_INVALID_ARG),
    (dict(), 1, dict(ws_bytes=16), M.MOE_ERR_CAPACITY),
    (dict(), 1, dict(out=None), M.MOE_ERR_INVALID_ARG),
    (dict(), 0, {}, M.MOE_OK),
    (dict(), 0, dict(x=None, out=None, ws=None, ws_bytes=0), M.MOE_OK),
])
def test_layer_refusals(lib, cfg, T, kw, code):
    a = dict(LAYER_OK, **kw)
    c = None if cfg is None else ctypes.byref(_cfg(**cfg))
    assert lib.moe_layer_fused(c, T, a["inter"], a["topk_idx"], a["topk_w"], a["x"], a["w13"], a["w13_scale"], a["w2"],
                               a["w2_scale"], a["ws"], a["ws_bytes"], a["out"], None) == code


def test_layer_workspace(lib):
    # a token mask per pair (8 bytes, the whole rounded up to 16) and a bf16 row of `inter` per pair
    assert M.moe_layer_workspace_bytes(_cfg(max_tokens=5, num_topk=3), 256) == 128 + 5 * 3 * 256 * 2
    assert M.moe_layer_workspace_bytes(_cfg(max_tokens=4096), 256) == 64 * 2 * 8 + 64 * 2 * 256 * 2
    assert M.moe_layer_workspace_bytes(_cfg(), 100) == 0
    assert M.moe_layer_workspace_bytes(_cfg(num_topk=0), 256) == 0
    need = M.moe_layer_workspace_bytes(_cfg(max_tokens=5, num_topk=3), 256)
    a = dict(LAYER_OK)
    c = _cfg(max_tokens=5, num_topk=3)
    assert lib.moe_layer_fused(ctypes.byref(c), 5, 256, a["topk_idx"], a["topk_w"], a["x"], a["w13"], a["w13_scale"],
                               a["w2"], a["w2_scale"], a["ws"], need - 1, a["out"], None) == M.MOE_ERR_CAPACITY


# ---- the reference itself --------------------------------------------------------------


@pytest.mark.parametrize("quant", [R.FP8_F32, R.FP8_UE8M0, R.MXFP8])
def test_reference_quantizer_matches_the_oracle(quant):
    """bf16 rows quantized by the 64-bit reference and by the oracle's dispatch: the same scales, and the same
    bytes except where x / s lies so near a rounding border that its fp32 quotient falls on the other side
    (none in power-of-two formats, whose quotients are exact)."""
    gen = torch.Generator().manual_seed(5)
    T, H = 64, 640
    x = torch.randn(T, H, generator=gen) * torch.exp2(torch.randint(-20, 20, (T, 1), generator=gen))
    x[3] = 0.0
    x[4, :128] = 448.0
    x[5, :128] = 449.0
    bits = x.bfloat16()
    ids = np.zeros((T, 1), np.int32)
    h = oracle.dispatch_layout(ids, 1, 1, 0, 1, 1, rows_cap=T)
    ox, osc, _ = oracle.dispatch(bits.view(torch.int16).numpy().view(np.uint16), h["pair_to_row"], 1, quant, T)
    q, s = R.quantize(bits, quant)
    got = s.numpy()
    want = np.ascontiguousarray(osc).view(got.dtype).reshape(got.shape)
    assert np.array_equal(got, want)
    differ = int((q.numpy() != np.ascontiguousarray(ox).view(np.uint8).reshape(T, H)).sum())
    assert differ <= (2 if quant == R.FP8_F32 else 0)


def test_reference_bounds_hold_for_a_rounded_product():
    """assert_bf16 accepts a correctly rounded result and refuses one that is a whole step off."""
    gen = torch.Generator().manual_seed(6)
    a, w = torch.randn(9, 256, generator=gen, dtype=R.D), torch.randn(40, 256, generator=gen, dtype=R.D)
    y, bound = R.product(a, w)
    R.assert_bf16(y.bfloat16(), y, bound * 0, "rounded")
    off = y.bfloat16()
    off[2, 3] = off[2, 3] * (1 + 2 ** -5)
    with pytest.raises(AssertionError):
        R.assert_bf16(off, y, bound * 0, "off")


def test_reference_rows_refuse_a_wrong_scale():
    x = torch.randn(4, 256, generator=torch.Generator().manual_seed(7), dtype=R.D)
    for quant in (R.FP8_F32, R.FP8_UE8M0, R.MXFP8):
        q, s = R.quantize(x, quant)
        R.assert_rows(q, s, x, x * 0, quant, "own")
        bad = s.clone()
        bad.view(-1)[0] = bad.view(-1)[0] * 2 if quant == R.FP8_F32 else bad.view(-1)[0] + 1
        with pytest.raises(AssertionError):
            R.assert_rows(q, bad, x, x * 0, quant, "wrong")
