"""More refusals of the operators of a whole prompt's experts on the host,
before any CUDA call."""

import pytest

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
