"""More refusals of the operators of a whole prompt's experts on the host,
before any CUDA call."""

import pytest
import torch

from tests.test_moe_host import INVALID, M, OK, lib  # noqa: F401


def test_experts_fault(M, lib):
    call = lib.msk_debug_experts_fault
    try:
        assert call(-2, 0) == INVALID and call(0, 200_000_001) == INVALID
        assert call(3, 1_000_000) == OK and call(0, 200_000_000) == OK
        with pytest.raises(ValueError):
            M.msk_debug_experts_fault(1 << 31)
        with pytest.raises(M.MskError):
            M.msk_debug_experts_fault(-7)
    finally:
        assert call(-1, 0) == OK


def test_slots_of_several_experts_a_token_need_top_k(M):
    """Without it every slot would be taken as a token, and those behind the last token as that one."""
    class W:
        n_experts, rows, cols, desc = 2, 8, 128, None
        _packed = torch.zeros(1)
    class X:
        rows, cols, desc = 5, 128, None
        _packed = torch.zeros(1)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="top_k"):
        M.msk_experts_fp4(X, W, off, slots=torch.zeros(10, dtype=torch.int32))
    for bad in (0, -1, 1 << 31):
        with pytest.raises(ValueError, match="top_k"):
            M.msk_experts_fp4(X, W, off, slots=torch.zeros(10, dtype=torch.int32), top_k=bad)
