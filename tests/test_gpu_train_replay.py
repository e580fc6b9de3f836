"""Every kernel of the bf16 expert layer captured once and replayed on changed
inputs, with eager work in between: each replay gives the bytes of the eager call,
and so does a call on another stream beside a second one.  Shapes reach the strips
of 16 and 32 rows, tiles of 64, 128 and 256 rows, rows kept in 8 bits, weight tiles
of both sizes, rows shared by several blocks, and the sums of an epilogue.
"""
import pytest
import torch

import combine_topk_idx_amd as M
from test_gpu_train import BF16, FP8, MX, UE8M0, Rows, _filled, _format_buffers, _gen, _gpu, _say, _weights  # noqa: F401

pytestmark = pytest.mark.gpu

EXPERTS = dict(T=150, E=5, K=2, layout="contiguous", align=16, holes=0.1, seed=8)


class Call:
    """An operator on buffers of its own: inputs() gives it values of a seed, run() calls it, outputs() are what it wrote."""

    def __init__(self, op, layout, n, k, save=None, **more):
        self.op, self.n, self.k, self.save, self.more = op, n, k, save, more
        self.rows = rows = Rows(H=n if op == "combine" else k, **layout)
        g, E, R = _gen(1), rows.E, rows.n + 2
        self.w = _weights(g, E, n, k) if op in ("gated", "linear", "grad_input") else None
        wide, fmt = (n if op == "act" else k), BF16 if save is None or op in ("gated", "linear") else save
        self.x = torch.empty(R, n if op in ("grad_input", "combine") else wide, dtype=torch.bfloat16, device="cuda")
        self.dy = torch.empty(R, n, dtype=torch.bfloat16, device="cuda")
        self.q, self.s = (self.x, None) if fmt == BF16 else _format_buffers(R, wide, fmt)
        self.bias = torch.empty(E, n, dtype=torch.bfloat16, device="cuda")
        self.dout = torch.empty(rows.T, n, dtype=torch.bfloat16, device="cuda")
        self.tw = torch.empty(rows.T, rows.cfg.num_topk, device="cuda")
        self.out = {}
        if op == "gated":
            self.out["h"] = _filled((R, n // 2), torch.bfloat16)
        if op == "linear":
            self.out["y"] = _filled((R, n), torch.bfloat16)
        if op in ("gated", "linear") and save is not None:
            self.out["saved"], self.out["scale"] = _format_buffers(R, n, save)
        if op == "grad_input":
            self.out["da"] = _filled((R, k), torch.bfloat16)
        if op == "grad_weight":
            self.out["dw"], self.out["db"] = _filled((E, n, k), torch.float32), _filled((E, n), torch.float32)
            size = M.moe_grad_weight_workspace_bytes(rows.cfg, rows.T, n, k)
            assert (size > 0) == more.get("shared", False)
            self.ws = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
        if op == "act":
            self.out["ds"], self.out["y"] = _filled((R, n), torch.bfloat16), _filled((R, n // 2), torch.bfloat16)
        if op == "combine":
            self.out["dy"], self.out["dw"] = _filled((R, n), torch.bfloat16), _filled(self.tw.shape, torch.float32)
        torch.cuda.synchronize()

    def inputs(self, seed):
        g = _gen(seed)
        for t in (self.x, self.dy, self.bias, self.dout):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        self.tw.copy_(torch.rand(self.tw.shape, generator=g, device="cuda"))
        if self.s is not None:
            self.q.copy_(torch.randint(0, 0x78, self.q.shape, generator=g, device="cuda"))
            if self.s.dtype == torch.float32:
                self.s.copy_(torch.rand(self.s.shape, generator=g, device="cuda"))
            else:
                b = self.s.view(torch.uint8)
                b.copy_(torch.randint(120, 125, b.shape, generator=g, device="cuda"))
        for name, t in self.out.items():
            if t is not None:
                if name in ("dw", "db"):
                    t.copy_(torch.randn(t.shape, generator=g, device="cuda"))  # what is added to
                else:
                    t.view(torch.uint8).fill_(0xA5)

    def run(self):
        r, n, k, o = self.rows, self.n, self.k, self.out
        save = BF16 if self.save is None else self.save
        if self.op == "gated":
            M.moe_ffn_gated(r.cfg, r.T, n // 2, M.ACT_SILU, self.x, self.w, r.handle, o["h"], o.get("saved"), o.get("scale"),
                            save)
        elif self.op == "linear":
            M.moe_expert_linear(r.cfg, r.T, n, k, M.ACT_GELU, self.x, self.w, self.bias, self.dy, r.handle, o["y"],
                                o.get("saved"), o.get("scale"), save)
        elif self.op == "grad_input":
            M.moe_expert_grad_input(r.cfg, r.T, n, k, self.x, self.w, r.handle, o["da"])
        elif self.op == "grad_weight":
            M.moe_expert_grad_weight(r.cfg, r.T, n, k, self.dy, self.q, self.s, save, r.handle, o["dw"], o["db"],
                                     self.more.get("accumulate", False), self.ws)
        elif self.op == "act":
            M.moe_activation_backward(r.cfg, r.T, n // 2, M.ACT_SILU, True, self.dy[:, :n // 2].contiguous(), self.q, self.s,
                                      save, r.handle, o["ds"], o["y"])
        else:
            M.moe_combine_backward(r.cfg, r.T, self.dout, self.dy, self.tw, r.handle, o["dy"], o["dw"])

    def outputs(self):
        return {name: t.clone() for name, t in self.out.items() if t is not None}


CALLS = {
    "gated strips of 16": ("gated", dict(T=9), 48, 1096),
    "gated strips of 32": ("gated", dict(T=30), 272, 584, BF16),
    "gated tiles of 64": ("gated", EXPERTS, 528, 264, BF16),
    "gated tiles of 64 kept in 8 bits": ("gated", dict(T=257), 768, 136, UE8M0),
    "gated tiles of 128": ("gated", dict(T=300), 13456, 72, BF16),
    "gated tiles of 256": ("gated", dict(T=310), 25600, 136, FP8),
    "linear strips of 16": ("linear", EXPERTS | dict(T=30), 40, 1096, BF16),
    "linear tiles of 64": ("linear", dict(T=257), 640, 264, MX),
    "linear tiles of 128": ("linear", dict(T=300), 13448, 72),
    "linear tiles of 256": ("linear", dict(T=310), 25608, 136),
    "input gradient, tiles of 64": ("grad_input", EXPERTS, 200, 264),
    "input gradient, tiles of 256": ("grad_input", dict(T=310), 72, 25608),
    "weights 128 x 256": ("grad_weight", EXPERTS, 264, 328),
    "weights 128 x 256 from 8 bits, added": ("grad_weight", EXPERTS, 264, 384, MX, dict(accumulate=True)),
    "weights with shared rows": ("grad_weight", dict(T=4097), 72, 136, None, dict(shared=True)),
    "weights with shared rows from 8 bits, added": ("grad_weight", dict(T=4097), 72, 256, FP8,
                                                    dict(shared=True, accumulate=True)),
    "weights 256 x 256, added": ("grad_weight", dict(T=1283), 2056, 4104, None, dict(accumulate=True)),
    "weights 256 x 256 from 8 bits": ("grad_weight", dict(T=1283), 2056, 4224, UE8M0),
    "activation": ("act", EXPERTS, 144, 8),
    "activation from 8 bits": ("act", EXPERTS, 512, 8, UE8M0),
    "combine": ("combine", EXPERTS, 264, 8),
}


def _call(name):
    op, layout, n, k, *rest = CALLS[name]
    save, more = (rest + [None, {}][len(rest):])[:2]
    return Call(op, layout, n, k, save, **more)


@pytest.mark.parametrize("name", CALLS)
def test_replayed(name):
    _say(f"replayed: {name}")
    c = _call(name)
    want = {}
    for seed in (1, 2):
        c.inputs(seed)
        c.run()
        torch.cuda.synchronize()
        want[seed] = c.outputs()
    assert any(not torch.equal(want[1][n].view(torch.uint8), want[2][n].view(torch.uint8)) for n in want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for seed in (2, 1, 1, 2):
        c.inputs(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = c.outputs()
        for n, v in want[seed].items():
            assert torch.equal(got[n].view(torch.uint8), v.view(torch.uint8)), (seed, n)
        c.run()  # eager work between the replays
        torch.cuda.synchronize()


@pytest.mark.parametrize("first,second", [
    ("weights with shared rows", "weights with shared rows from 8 bits, added"),
    ("gated tiles of 256", "linear tiles of 256"),
    ("weights 256 x 256, added", "gated strips of 16"),
    ("weights 128 x 256 from 8 bits, added", "combine"),
])
def test_two_at_once(first, second):
    """Calls on two streams, each with its own buffers and workspace."""
    _say(f"two at once: {first}, {second}")
    calls = [_call(first), _call(second)]
    want = []
    for c in calls:
        c.inputs(3)
        c.run()
        torch.cuda.synchronize()
        want.append(c.outputs())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for c in calls:
            c.inputs(3)
        torch.cuda.synchronize()
        for s, c in zip(streams, calls):
            with torch.cuda.stream(s):
                c.run()
        torch.cuda.synchronize()
        for c, w in zip(calls, want):
            for n, v in c.outputs().items():
                assert torch.equal(v.view(torch.uint8), w[n].view(torch.uint8)), n
