"""Weight gradients at both tile sizes, on either side of the rule that chooses.

256 x 256 tiles take over when rounds over the compute units and rows per expert
make them the faster ones; these cases have enough rows for them, with channels
that end inside a tile, rows that end inside a step, steps that are no multiple
of a round of four, an expert without rows, and more tiles than compute units.
Each has a neighbour with fewer rows or tiles that takes 128 x 256.
"""
import pytest
import torch

import combine_topk_idx_amd as M
import strict_reference as S
import train_reference as R
from test_gpu_train import (BF16, D, FP8, MX, UE8M0, Rows, _filled, _gen, _gpu, _grad_weight,  # noqa: F401
                            _grad_weight_reference, _say, _untouched)

pytestmark = pytest.mark.gpu

LAYOUTS = {
    "dense1283": dict(T=1283),                # 41 steps, the last one of 3 rows
    "dense1153": dict(T=1153),                # 37 steps, one row in the last
    "dense300": dict(T=300),                  # too few rows
    "experts": dict(T=1500, E=5, K=3, layout="contiguous", align=1, used=4, holes=0.05, seed=1),    # one without rows
    "slab": dict(T=1400, E=3, K=2, layout="masked", capacity=901, seed=2),       # drops pairs
    "short": dict(T=200, E=5, K=3, layout="contiguous", align=16, used=4, seed=3),
}


@pytest.mark.parametrize("layout,n,k,quant,dtype,bias", [
    ("dense1283", 2056, 4104, BF16, torch.float32, True),
    ("dense1283", 2056, 4104, BF16, torch.bfloat16, False),
    ("dense1153", 2312, 3720, BF16, torch.bfloat16, True),
    ("dense1283", 2056, 4224, FP8, torch.float32, True),
    ("dense1153", 2056, 4224, UE8M0, torch.bfloat16, True),
    ("dense1283", 2056, 4224, MX, torch.float32, False),
    ("dense1153", 2312, 3712, MX, torch.bfloat16, True),
    ("experts", 1032, 1800, BF16, torch.float32, True),
    ("experts", 1032, 1920, UE8M0, torch.float32, True),
    ("experts", 1288, 1800, BF16, torch.bfloat16, True),
    ("experts", 1032, 1664, FP8, torch.bfloat16, True),
    ("slab", 1032, 2568, BF16, torch.bfloat16, True),
    ("slab", 1544, 1920, MX, torch.float32, True),
    # more tiles than compute units
    ("experts", 1288, 4104, BF16, torch.bfloat16, True),
    ("experts", 1288, 4224, FP8, torch.float32, True),
    # 128 x 256: too few rows, too few tiles, or a second round that is nearly empty
    ("dense300", 2056, 4104, BF16, torch.float32, True),
    ("dense300", 2056, 4224, UE8M0, torch.float32, True),
    ("dense1283", 2048, 2048, BF16, torch.bfloat16, True),
    ("dense1283", 4096, 4352, MX, torch.bfloat16, True),
    ("dense1283", 4096, 4352, FP8, torch.bfloat16, True),
    ("short", 1032, 4104, BF16, torch.float32, True),
    ("short", 1032, 4224, MX, torch.bfloat16, True),
])
def test_grad_weight(layout, n, k, quant, dtype, bias):
    _say(f"grad weight tiles {layout} n={n} k={k} quant={quant} {dtype} bias={bias}")
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
            S.assert_bf16(dw[e], v, b, f"dw[{e}]")
        if bias:
            R.assert_near(db[e], sv, sb, f"dbias[{e}]")
    _untouched(dw[rows.E], "dw behind the last expert")
    if bias:
        _untouched(db[rows.E], "dbias behind the last expert")


@pytest.mark.parametrize("layout,n,k,quant", [("dense1283", 2056, 4104, BF16), ("experts", 1032, 1800, BF16),
                                              ("experts", 1288, 4224, UE8M0), ("short", 1032, 4104, BF16)])
def test_grad_weight_accumulates(layout, n, k, quant):
    _say(f"grad weight tiles accumulates {layout} n={n} k={k} quant={quant}")
    rows = Rows(**LAYOUTS[layout])
    g = _gen(n)
    dy = rows.input(g, n)
    q, s = rows.formatted(g, k, quant)
    was, bwas = torch.randn(rows.E, n, k, generator=g, device="cuda") * 3, torch.randn(rows.E, n, generator=g, device="cuda")
    dw, db = was.clone(), bwas.clone()
    _grad_weight(rows, n, k, dy, q, s, quant, dw, db, accumulate=True)
    for e, (v, b), (sv, sb) in _grad_weight_reference(rows, dy, q, s, quant):
        lo, hi = rows.spans[e]
        if lo == hi:
            assert torch.equal(dw[e], was[e]) and torch.equal(db[e], bwas[e])
        old, bold = was[e].to(D), bwas[e].to(D)
        R.assert_near(dw[e], old + v, b + (old.abs() + v.abs()) * 2.0 ** -23, "dw")
        R.assert_near(db[e], bold + sv, sb + (bold.abs() + sv.abs()) * 2.0 ** -23, "dbias")


@pytest.mark.parametrize("T,n,k,shared", [(1100, 64, 32768, True), (1100, 136, 16384, True), (1100, 64, 33024, False),
                                          (500, 64, 32768, False)])
def test_rows_are_shared_up_to_half_the_compute_units(T, n, k, shared):
    """128 tiles of weights share their rows between two blocks each from 1024 rows on, 129 do not (256 compute units)."""
    _say(f"grad weight shared rows T={T} n={n} k={k}")
    rows = Rows(T)
    size = M.moe_grad_weight_workspace_bytes(rows.cfg, T, n, k)
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert size == (2 * (n * k + n) * 4 if shared else 0)
    g = _gen(k)
    dy, a = rows.input(g, n, 0.02), rows.input(g, k)
    dw, db = _filled((2, n, k), torch.float32), _filled((2, n), torch.float32)
    _grad_weight(rows, n, k, dy, a, None, BF16, dw, db)
    for _, (v, b), (sv, sb) in _grad_weight_reference(rows, dy, a, None, BF16):
        R.assert_near(dw[0], v, b, "dw")
        R.assert_near(db[0], sv, sb, "dbias")
    _untouched(dw[1], "dw behind the last expert")
    _untouched(db[1], "dbias behind the last expert")


@pytest.mark.parametrize("quant", [BF16, UE8M0])
def test_tiles_agree_on_shared_channels(quant):
    """The first 256 x 512 weights of a large product and the same ones alone: other tiles, the same bits, for each sums
    its rows in the same order (1000 rows are too few to be shared among blocks)."""
    _say(f"grad weight tiles agree quant={quant}")
    T, n, k = 1000, 2304, 4096
    rows = Rows(T)
    g = _gen(9)
    dy = rows.input(g, n)
    q, s = rows.formatted(g, k, quant)
    dw, db = _filled((1, n, k), torch.float32), _filled((1, n), torch.float32)
    _grad_weight(rows, n, k, dy, q, s, quant, dw, db)
    a, b = dy[:, :256].contiguous(), q[:, :512].contiguous()
    sc = None if s is None else s[:, :1].contiguous()
    part, pb = _filled((1, 256, 512), torch.float32), _filled((1, 256), torch.float32)
    assert M.moe_grad_weight_workspace_bytes(rows.cfg, T, 256, 512) == 0
    _grad_weight(rows, 256, 512, a, b, sc, quant, part, pb)
    assert torch.equal(part[0], dw[0, :256, :512]) and torch.equal(pb[0], db[0, :256])
