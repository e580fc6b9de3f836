"""The compiled code of the bf16 products along every way through it (no GPU
needed): sums in accumulators and in vector registers, operands, what starts a
sum, and loops that stay free of spilled registers.  codegen_ways has the rules;
mistakes are planted in small pieces of code to show that they are found."""
import os
import re
import subprocess

import pytest

import codegen_ways as W
import test_train_codegen
from combine_topk_idx_amd import build as B


def test_the_compiled_code_is_that_of_the_build(monkeypatch):
    """The options are build()'s, here and where they are written out."""
    seen = []

    def run(cmd, **kw):
        seen.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "")

    monkeypatch.setattr(B.subprocess, "run", run)
    with pytest.raises(RuntimeError):
        B.build()
    assert seen[0][1:1 + len(B.OPTIONS)] == B.OPTIONS
    assert not [x for x in seen[0][1 + len(B.OPTIONS):] if x.startswith(("-m", "-f", "-O", "-X", "-D"))]
    assert test_train_codegen.OPTIONS == B.OPTIONS


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    out = tmp_path_factory.mktemp("s")
    running = [(f, subprocess.Popen([B.hipcc(), *B.OPTIONS, "-S", "--cuda-device-only", "-o", str(out / f) + ".s",
                                     os.path.join(B.PKG, "csrc", f)], stderr=subprocess.DEVNULL))
               for f in test_train_codegen.FILES]
    found = {}
    for f, p in running:
        assert p.wait(timeout=600) == 0
        found.update(W.parse(open(str(out / f) + ".s").read()))
    return found


def test_no_hazard_on_any_way(kernels):
    inline = 0
    for name, kernel in kernels.items():
        inline += sum(kernel[0][i].startswith("v_mfma") for i in kernel[2])
        assert not W.hazards(kernel), name
    assert inline > 3000


def test_loops_that_multiply_do_not_spill(kernels):
    """No scratch access in a tile's loop, and no wait for every load but the kernels' own: a reload waits for all loads
    before it, whole stages that the loop's counted waits leave on their way."""
    seen = 0
    for name, kernel in kernels.items():
        if "tiles" not in name:
            continue
        inner = W.loops(kernel)
        assert inner, name
        for blocks in inner:
            seen += 1
            for first, last in blocks:
                idle = False  # no load since a wait for all of them
                for i in range(first, last + 1):
                    x = kernel[0][i]
                    assert not x.startswith("scratch_"), f"{name}: {x}"
                    if re.match(r"s_waitcnt .*vmcnt\(0\)", x):
                        own = "lgkmcnt(0)" in x and kernel[0][i + 1].startswith("s_barrier")
                        assert own or idle, f"{name}: {x}"
                        idle = True
                    elif x.startswith(("buffer_", "global_")):
                        idle = False
    assert seen >= 40


# ---- mistakes that have to be found ------------------------------------------------------------


def _kernel(body):
    return W.parse("_ZNplanted:  ; @planted\n" + body + "\n\ts_endpgm\n.Lfunc_end0:\n")["_ZNplanted"]


SUM = "\t;;#ASMSTART\n\tv_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[8:11], a[0:3]\n\t;;#ASMEND\n"
BESIDE = "\t;;#ASMSTART\n\ts_nop 1\n\tv_mfma_f32_16x16x32_bf16 v[0:3], v[4:7], v[8:11], v[0:3]\n\t;;#ASMEND\n"
WAIT = "\ts_nop 15\n\ts_nop 7\n"
TURN = ("\t;;#ASMSTART\n\ts_cmp_lt_i32 s0, s1\n\ts_cbranch_scc1 .Lturn0\n" + WAIT + ".Lturn0:\n\t;;#ASMEND\n")
BACK = "\ts_cmp_ge_i32 s0, s1\n\ts_cbranch_scc0 .LBB0_1\n"
READ = "\tv_accvgpr_read_b32 v20, a2\n"


@pytest.mark.parametrize("body", [
    SUM + SUM + WAIT + READ,                                   # sums add up in place
    BESIDE + BESIDE + WAIT + "\tscratch_store_dword off, v1, off\n",
    ".LBB0_1:\n" + SUM + TURN + BACK + READ,                   # the last turn has waited
    ".LBB0_1:\n" + SUM + TURN + "\ts_addk_i32 s5, 0x80\n" + BACK.replace("ge", "lt").replace("scc0", "scc1") + READ,
    "\tv_accvgpr_write_b32 a0, 0\n\ts_nop 1\n" + SUM,
    "\tv_mov_b32_e32 v1, 0\n" + BESIDE,                        # has its own pause
    "\tv_mov_b32_e32 v12, v4\n" + SUM,                         # reads an operand
])
def test_code_without_a_mistake(body):
    assert not W.hazards(_kernel(body))


@pytest.mark.parametrize("body", [
    SUM + READ,                                                # a sum is read at once
    SUM + "\ts_nop 15\n" + READ,                               # too soon
    SUM + "\tv_accvgpr_write_b32 a3, 0\n",                     # or written
    SUM + "\tv_mfma_f32_16x16x32_bf16 a[4:7], v[4:7], a[0:3], a[4:7]\n",   # or multiplied
    BESIDE + "\tv_add_f32_e32 v12, v1, v1\n",                  # the same for sums in vector registers
    BESIDE + "\tscratch_store_dword off, v1, off\n",
    BESIDE + "\tv_mov_b32_e32 v30, v0\n",
    BESIDE + "\tbuffer_load_dword v2, v40, s[0:3], 0 offen\n",
    ".LBB0_1:\n" + SUM + TURN + READ + BACK,                   # between the wait of the last turn and the branch back
    ".LBB0_1:\n" + SUM + TURN + BACK.replace("s1", "s2") + READ,           # a branch that compares something else
    ".LBB0_1:\n" + READ + SUM + TURN + BACK,                   # at the head of the next turn
    ".LBB0_1:\n" + SUM + TURN + "\ts_cmp_ge_i32 s0, s1\n\ts_cbranch_scc1 .LBB0_2\n" + READ + "\ts_branch .LBB0_1\n.LBB0_2:\n",
    "\tv_accvgpr_write_b32 a0, 0\n" + SUM,                     # what a sum starts from
    "\tv_accvgpr_write_b32 a3, 0\n\ts_nop 0\n" + SUM,
    "\tv_add_u32_e32 v11, v12, v13\n" + SUM,                   # an operand
    "\tv_mov_b32_e32 v4, 0\n\ts_branch .LBB0_5\n.LBB0_5:\n" + SUM,         # on the way from another block
    "\ts_cbranch_vccz .LBB0_5\n\tv_mov_b32_e32 v4, 0\n.LBB0_5:\n" + SUM,
])
def test_planted_mistakes_are_found(body):
    assert W.hazards(_kernel(body))
