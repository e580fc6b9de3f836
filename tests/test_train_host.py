"""Host-side tests of the bf16 expert layer and its gradients (no GPU needed):
the header, exported symbols, workspace sizes, every refusal of the C ABI
(decided before anything is enqueued; pointers are fake aligned addresses), and
the 64-bit reference against differences."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import combine_topk_idx_amd as M
import train_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_train.h")
FAKE = 0x7F0000000000  # never dereferenced
NAMES = ["moe_activation_backward", "moe_combine_backward", "moe_expert_grad_input", "moe_expert_grad_weight",
         "moe_expert_linear", "moe_ffn_gated", "moe_grad_weight_workspace_bytes"]
BAD, CAP, UNS, OK = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_CAPACITY, M.MOE_ERR_UNSUPPORTED, M.MOE_OK


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.LIB_PATH):
        pytest.fail("libmoe_dispatch.so is not built (python -m combine_topk_idx_amd.build)")
    return M.library()


def _cfg(**kw):
    base = dict(max_tokens=64, hidden=256, num_experts=8, num_topk=2, num_ranks=2,
                layout=M.LAYOUT_CONTIGUOUS, align=1, capacity=1, quant=M.QUANT_NONE, num_cus=0)
    base.update(kw)
    return M.MoeConfig(**base)


def _cfgp(cfg):
    return None if cfg is None else ctypes.byref(_cfg(**cfg))


def _handle(h):
    if h is None:
        return None
    vals = {n: FAKE + 0x1000 * i for i, (n, _) in enumerate(M.MoeHandle._fields_)}
    vals.update(h)
    return ctypes.byref(M.MoeHandle(**vals))


def test_header_declares_and_library_exports(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(moe_[a-z_]+)\s*\(", src))) == NAMES
    out = subprocess.run(["nm", "-D", "--defined-only", M.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r"\bT (moe_[a-z_]+)\b", out))
    assert not [n for n in NAMES if n not in exported]


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "moe_train.h"\nint main(void) { return MOE_ACT_RELU != 3; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    "-fsyntax-only", str(src)], check=True)


# What every entry point refuses of its config, tokens and handle.
COMMON = [
    (None, 1, {}, BAD),
    (dict(num_topk=0), 1, {}, BAD),
    (dict(hidden=12), 1, {}, BAD),
    (dict(), -1, {}, BAD),
    (dict(), 65, {}, CAP),
    (dict(), 1, dict(handle=dict(recv_count=None)), BAD),
    (dict(), 1, dict(handle=dict(expert_offset=FAKE + 2)), BAD),
    (dict(), 1, dict(handle=None), BAD),                       # dense needs one expert
    (dict(), 0, {}, OK),
]


def _gated(lib, cfg, T, **kw):
    a = dict(inter=256, act=1, a=FAKE, w=FAKE, handle={}, h=FAKE, saved=FAKE, scale=FAKE, quant=M.QUANT_FP8_F32)
    a.update(kw)
    return lib.moe_ffn_gated(_cfgp(cfg), T, a["inter"], a["act"], a["a"], a["w"], _handle(a["handle"]), a["h"],
                             a["saved"], a["scale"], a["quant"], None)


@pytest.mark.parametrize("cfg,T,kw,code", COMMON + [
    (dict(), 1, dict(inter=0), BAD),
    (dict(), 1, dict(inter=-128), BAD),
    (dict(), 1, dict(inter=12), BAD),
    (dict(), 1, dict(inter=136), BAD),                         # 8-bit rows need whole blocks
    (dict(), 0, dict(inter=136), BAD),
    (dict(), 1, dict(inter=(1 << 19) + 8), UNS),
    (dict(hidden=(1 << 20) + 8), 1, {}, UNS),
    (dict(), 1, dict(act=-1), BAD),
    (dict(), 1, dict(act=4), BAD),
    (dict(), 1, dict(quant=4), BAD),
    (dict(), 1, dict(quant=-1, saved=None, scale=None), BAD),
    (dict(), 1, dict(saved=None), BAD),                        # scales without rows
    (dict(), 1, dict(scale=None), BAD),
    (dict(), 1, dict(quant=M.QUANT_NONE), BAD),                # bf16 rows have no scales
    (dict(), 1, dict(saved=FAKE + 8), BAD),
    (dict(), 1, dict(scale=FAKE + 2), BAD),
    (dict(), 1, dict(a=None), BAD),
    (dict(), 1, dict(a=FAKE + 8), BAD),
    (dict(), 1, dict(w=None), BAD),
    (dict(), 1, dict(w=FAKE + 2), BAD),
    (dict(), 1, dict(h=None), BAD),
    (dict(), 1, dict(h=FAKE + 4), BAD),
    (dict(), 0, dict(a=None, w=None, h=None, saved=None, scale=None), OK),
    (dict(num_experts=1, num_topk=1, num_ranks=1), 0, dict(handle=None), OK),
])
def test_gated_refusals(lib, cfg, T, kw, code):
    assert _gated(lib, cfg, T, **kw) == code


def _linear(lib, cfg, T, **kw):
    a = dict(n=256, k=256, act=0, a=FAKE, w=FAKE, bias=FAKE, residual=FAKE, handle={}, y=FAKE, saved=FAKE, scale=FAKE,
             quant=M.QUANT_MXFP8)
    a.update(kw)
    return lib.moe_expert_linear(_cfgp(cfg), T, a["n"], a["k"], a["act"], a["a"], a["w"], a["bias"], a["residual"],
                                 _handle(a["handle"]), a["y"], a["saved"], a["scale"], a["quant"], None)


@pytest.mark.parametrize("cfg,T,kw,code", COMMON + [
    (dict(), 1, dict(n=0), BAD),
    (dict(), 1, dict(n=12), BAD),
    (dict(), 1, dict(n=136), BAD),
    (dict(), 1, dict(k=0), BAD),
    (dict(), 1, dict(k=-8), BAD),
    (dict(), 1, dict(k=4), BAD),
    (dict(), 1, dict(n=(1 << 20) + 128), UNS),
    (dict(), 1, dict(k=(1 << 20) + 8), UNS),
    (dict(), 1, dict(act=7), BAD),
    (dict(), 1, dict(quant=9), BAD),
    (dict(), 1, dict(saved=None), BAD),
    (dict(), 1, dict(scale=None), BAD),
    (dict(), 1, dict(a=None), BAD),
    (dict(), 1, dict(w=None), BAD),
    (dict(), 1, dict(w=FAKE + 8), BAD),
    (dict(), 1, dict(bias=FAKE + 2), BAD),
    (dict(), 1, dict(residual=FAKE + 8), BAD),
    (dict(), 1, dict(y=None), BAD),
    (dict(), 1, dict(y=FAKE + 8), BAD),
    (dict(), 0, dict(a=None, w=None, bias=None, residual=None, y=None, saved=None, scale=None), OK),
])
def test_linear_refusals(lib, cfg, T, kw, code):
    assert _linear(lib, cfg, T, **kw) == code


def _act(lib, cfg, T, **kw):
    a = dict(n=256, act=1, gated=1, dy=FAKE, saved=FAKE, scale=FAKE, quant=M.QUANT_FP8_UE8M0, handle={}, ds=FAKE, y=FAKE)
    a.update(kw)
    return lib.moe_activation_backward(_cfgp(cfg), T, a["n"], a["act"], a["gated"], a["dy"], a["saved"], a["scale"],
                                       a["quant"], _handle(a["handle"]), a["ds"], a["y"], None)


@pytest.mark.parametrize("cfg,T,kw,code", COMMON + [
    (dict(), 1, dict(n=0), BAD),
    (dict(), 1, dict(n=20), BAD),
    (dict(), 1, dict(n=136), BAD),
    (dict(), 1, dict(n=(1 << 19) + 128), UNS),
    (dict(), 1, dict(n=(1 << 20) + 128, gated=0), UNS),
    (dict(), 1, dict(gated=2), BAD),
    (dict(), 1, dict(act=-1), BAD),
    (dict(), 1, dict(quant=5), BAD),
    (dict(), 1, dict(dy=None), BAD),
    (dict(), 1, dict(dy=FAKE + 8), BAD),
    (dict(), 1, dict(saved=None), BAD),
    (dict(), 1, dict(saved=FAKE + 8), BAD),
    (dict(), 1, dict(scale=None), BAD),
    (dict(), 1, dict(quant=M.QUANT_NONE), BAD),                # bf16 rows have no scales
    (dict(), 1, dict(ds=None), BAD),
    (dict(), 1, dict(ds=FAKE + 2), BAD),
    (dict(), 1, dict(y=FAKE + 2), BAD),
    (dict(), 0, dict(dy=None, saved=None, scale=None, ds=None, y=None), OK),
])
def test_activation_backward_refusals(lib, cfg, T, kw, code):
    assert _act(lib, cfg, T, **kw) == code


def _grad_input(lib, cfg, T, **kw):
    a = dict(n=256, k=256, dy=FAKE, w=FAKE, handle={}, da=FAKE)
    a.update(kw)
    return lib.moe_expert_grad_input(_cfgp(cfg), T, a["n"], a["k"], a["dy"], a["w"], _handle(a["handle"]), a["da"], None)


@pytest.mark.parametrize("cfg,T,kw,code", COMMON + [
    (dict(), 1, dict(n=4), BAD),
    (dict(), 1, dict(k=9), BAD),
    (dict(), 1, dict(n=(1 << 20) + 8), UNS),
    (dict(), 1, dict(k=(1 << 20) + 8), UNS),
    (dict(), 1, dict(dy=None), BAD),
    (dict(), 1, dict(dy=FAKE + 8), BAD),
    (dict(), 1, dict(w=None), BAD),
    (dict(), 1, dict(w=FAKE + 8), BAD),
    (dict(), 1, dict(da=None), BAD),
    (dict(), 1, dict(da=FAKE + 8), BAD),
    (dict(), 0, dict(dy=None, w=None, da=None), OK),
])
def test_grad_input_refusals(lib, cfg, T, kw, code):
    assert _grad_input(lib, cfg, T, **kw) == code


def _grad_weight(lib, cfg, T, **kw):
    a = dict(n=256, k=256, dy=FAKE, a=FAKE, scale=FAKE, quant=M.QUANT_FP8_F32, handle={}, dw=FAKE, bf16=0, db=FAKE, acc=0,
             ws=FAKE, bytes=1 << 40)
    a.update(kw)
    return lib.moe_expert_grad_weight(_cfgp(cfg), T, a["n"], a["k"], a["dy"], a["a"], a["scale"], a["quant"],
                                      _handle(a["handle"]), a["dw"], a["bf16"], a["db"], a["acc"], a["ws"], a["bytes"],
                                      None)


DENSE = dict(max_tokens=8192, num_experts=1, num_topk=1, num_ranks=1)


@pytest.mark.parametrize("cfg,T,kw,code", [c for c in COMMON if c[3] != OK] + [
    (dict(), 1, dict(n=4), BAD),
    (dict(), 1, dict(k=0), BAD),
    (dict(), 1, dict(k=136), BAD),                             # 8-bit rows need whole blocks
    (dict(), 0, dict(k=136), BAD),
    (dict(), 1, dict(n=(1 << 20) + 8), UNS),
    (dict(), 1, dict(k=(1 << 20) + 128), UNS),
    (dict(), 1, dict(quant=4), BAD),
    (dict(), 1, dict(bf16=2), BAD),
    (dict(), 1, dict(acc=-1), BAD),
    (dict(), 1, dict(bf16=1, acc=1), BAD),                     # only fp32 gradients are added to
    (dict(), 1, dict(dy=None), BAD),
    (dict(), 1, dict(dy=FAKE + 8), BAD),
    (dict(), 1, dict(a=None), BAD),
    (dict(), 1, dict(a=FAKE + 8), BAD),
    (dict(), 1, dict(scale=None), BAD),
    (dict(), 1, dict(quant=M.QUANT_NONE), BAD),                # bf16 rows have no scales
    (dict(), 1, dict(dw=None), BAD),
    (dict(), 0, dict(dw=None), BAD),                           # zeros have to go somewhere
    (dict(), 1, dict(dw=FAKE + 8), BAD),
    (dict(), 1, dict(db=FAKE + 2), BAD),
    (DENSE, 8192, dict(handle=None, ws=None), BAD),
    (DENSE, 8192, dict(handle=None, ws=FAKE + 4), BAD),
    (DENSE, 8192, dict(handle=None, bytes=1024), CAP),
])
def test_grad_weight_refusals(lib, cfg, T, kw, code):
    assert _grad_weight(lib, cfg, T, **kw) == code


def _combine(lib, cfg, T, **kw):
    a = dict(dout=FAKE, y=FAKE, w=FAKE, handle={}, dy=FAKE, dw=FAKE)
    a.update(kw)
    return lib.moe_combine_backward(_cfgp(cfg), T, a["dout"], a["y"], a["w"], _handle(a["handle"]), a["dy"], a["dw"], None)


@pytest.mark.parametrize("cfg,T,kw,code", COMMON + [
    (dict(num_experts=1, num_topk=1, num_ranks=1), 1, dict(handle=None), BAD),
    (dict(), 1, dict(handle=dict(pair_to_row=FAKE + 1)), BAD),
    (dict(), 1, dict(dout=None), BAD),
    (dict(), 1, dict(dout=FAKE + 8), BAD),
    (dict(), 1, dict(y=None), BAD),                            # the weights' gradient needs it
    (dict(), 1, dict(dw=None), BAD),
    (dict(), 1, dict(y=FAKE + 8), BAD),
    (dict(), 1, dict(w=None), BAD),
    (dict(), 1, dict(w=FAKE + 2), BAD),
    (dict(), 1, dict(dy=None), BAD),
    (dict(), 1, dict(dy=FAKE + 8), BAD),
    (dict(), 1, dict(dw=FAKE + 2), BAD),
    (dict(), 0, dict(dout=None, y=None, w=None, dy=None, dw=None), OK),
])
def test_combine_backward_refusals(lib, cfg, T, kw, code):
    assert _combine(lib, cfg, T, **kw) == code


def test_workspace_sizes(lib):
    size = lambda T, n, k, **kw: M.moe_grad_weight_workspace_bytes(_cfg(**kw), T, n, k)  # noqa: E731
    assert size(64, 256, 256) == 0                             # few rows
    assert size(8192, 4096, 7168, max_tokens=8192) == 0        # many weights
    parts = size(8192, 256, 256, **DENSE)
    assert parts > 0 and parts % ((256 * 256 + 256) * 4) == 0
    for T in (0, 1, 100, 1000, 4096):                          # more tokens never need less
        assert size(T, 256, 256, **DENSE) <= parts
    assert size(8193, 256, 256, **DENSE) == 0                  # refused arguments
    assert size(-1, 256, 256, **DENSE) == 0
    assert size(64, 252, 256, **DENSE) == 0
    assert size(64, 256, (1 << 20) + 8, **DENSE) == 0


@pytest.mark.parametrize("kind", [R.NONE, R.SILU, R.GELU, R.RELU])
def test_reference_slopes_against_differences(kind):
    """The reference's gradients (64 bits) against central differences."""
    g = torch.Generator().manual_seed(kind)
    v = torch.randn(64, 48, generator=g, dtype=R.D) * 2
    v = torch.where(v.abs() < 1e-3, v + 0.01, v)  # relu has no slope at 0
    dy = torch.randn(64, 24, generator=g, dtype=R.D)
    d = torch.randn(64, 48, generator=g, dtype=R.D)
    (ds, _), _ = R.act_grads(dy, v, kind, True)
    loss = lambda x: (dy * R.gated(x, torch.zeros_like(x), kind)[0]).sum()  # noqa: E731
    h = 1e-6
    diff = (loss(v + h * d) - loss(v - h * d)) / (2 * h)
    # third-order remainder h^2 / 6 |f'''| |d|^3 and 2^-52 |loss| / h of rounding
    assert abs(float(diff - (ds * d).sum())) < 1e-4
