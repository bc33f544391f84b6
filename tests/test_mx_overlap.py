"""moe_pack_scales_mx is not done in place: overlapping buffers are refused (no GPU)."""
import ctypes

import pytest

from tests.test_abi import moe  # noqa: F401  (the built library)

BASE, SIZE = 1 << 20, 2 * 128 * 384 // 32


@pytest.mark.parametrize("at", [0, 16, -16, SIZE - 16, 16 - SIZE])
def test_overlap_is_refused(moe, at):
    st = moe._lib.moe_pack_scales_mx(2, 128, 384, 0, ctypes.c_void_p(BASE), ctypes.c_void_p(BASE + at), None)
    assert st == moe.MOE_ERR_INVALID_ARG
