"""Sizes at which the expert-layer operators refuse a call (no GPU needed: the
refusal comes before anything is enqueued, pointers are fake aligned addresses)."""
import ctypes

import pytest

import combine_topk_idx_amd as M

FAKE = 0x7F0000000000  # never dereferenced
TOP = 1 << 27


def _call(T, hidden, inter):
    c = M.MoeConfig(max_tokens=1, hidden=hidden, num_experts=1, num_topk=1, num_ranks=1, layout=M.LAYOUT_CONTIGUOUS,
                    align=1, capacity=1, quant=M.QUANT_FP8_F32)
    code = M.library().moe_layer_fused(ctypes.byref(c), T, inter, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                       1 << 40, FAKE, None)
    return code, M.moe_layer_workspace_bytes(c, inter)


@pytest.mark.parametrize("hidden,inter", [(128, TOP + 128), (128, 1 << 30), (TOP + 128, 128), (1 << 30, 128)])
def test_layer_refuses_more_channels_than_its_grids_hold(hidden, inter):
    assert _call(0, hidden, inter) == (M.MOE_ERR_UNSUPPORTED, 0)


@pytest.mark.parametrize("hidden,inter", [(128, TOP), (TOP, 128)])
def test_layer_takes_the_largest_sizes(hidden, inter):
    assert _call(0, hidden, inter) == (M.MOE_OK, 16 + 2 * inter)
