"""Limits of the bf16 layer's C ABI that every entry point shares (no GPU
needed; decided before anything is enqueued, pointers are fake aligned addresses)."""
import ctypes

import pytest

import combine_topk_idx_amd as M

FAKE = 0x7F0000000000  # never dereferenced


def _cfg(**kw):
    base = dict(max_tokens=64, hidden=256, num_experts=8, num_topk=2, num_ranks=2)
    base.update(kw)
    return M.MoeConfig(**base)


def _handle():
    return ctypes.byref(M.MoeHandle(*(FAKE + 0x1000 * i for i in range(len(M.MoeHandle._fields_)))))


@pytest.mark.parametrize("tokens", [0, 1])
@pytest.mark.parametrize("hidden", [(1 << 20) + 8, (1 << 30), (1 << 31) - 8])
def test_combine_backward_refuses_wide_rows(hidden, tokens):
    """More than MOE_TRAIN_MAX_CHANNELS channels, up to the largest that an int32 holds."""
    code = M.library().moe_combine_backward(ctypes.byref(_cfg(hidden=hidden)), tokens, FAKE, FAKE, FAKE, _handle(), FAKE,
                                            FAKE, None)
    assert code == M.MOE_ERR_UNSUPPORTED


def test_combine_backward_takes_the_widest_rows():
    """An empty batch of rows that are just as wide as allowed."""
    code = M.library().moe_combine_backward(ctypes.byref(_cfg(hidden=1 << 20)), 0, FAKE, FAKE, FAKE, _handle(), FAKE,
                                            FAKE, None)
    assert code == M.MOE_OK
