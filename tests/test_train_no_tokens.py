"""Workspaces of the training step for no tokens: a valid number, which the queries and the binding take (no GPU needed)."""
import pytest

from tests.test_abi import moe  # noqa: F401


@pytest.mark.parametrize("H", [8, 7168, 8192, 16384, 32768])
def test_norm_backward(moe, H):  # noqa: F811
    none, one = (moe.moe_workspace_bytes_norm_backward(T, H) for T in (0, 1))
    assert 0 < none <= one
    assert moe.workspace_norm_backward(0, H, device="cpu").numel() == none
    assert moe.moe_workspace_bytes_norm_backward(-1, H) == 0 and moe.moe_workspace_bytes_norm_backward(0, H + 1) == 0


def test_grouped(moe):  # noqa: F811
    cfg = dict(hidden=128, num_experts=8, top_k=2, intermediate=256, block_size=8)
    assert moe.workspace_grouped(cfg, 0, device="cpu").numel() == moe.moe_workspace_bytes_grouped(cfg, 0) > 0
