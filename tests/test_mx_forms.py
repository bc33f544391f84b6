"""Which form moe_expert_ffn_mx takes, and its workspace, by the rows that an expert holds (no GPU)."""
import pytest

from tests.test_abi import moe  # noqa: F401  (the built library)

LAYER = dict(hidden=2048, num_experts=128, top_k=8, intermediate=768, block_size=16)


@pytest.mark.parametrize("T,rows", [(1, 32), (256, 32), (257, 128), (1535, 128), (1536, 256), (8192, 256)])
def test_form_of_token_choice(moe, T, rows):
    assert moe.moe_expert_ffn_mx_tile_rows(LAYER, T) == rows


@pytest.mark.parametrize("cf,scale", [(0.0, 1), (1.0, 1), (2.0, 2)])
@pytest.mark.parametrize("T,rows", [(96, 32), (256, 32), (258, 128), (1520, 128), (1536, 256), (8192, 256)])
def test_form_of_expert_choice(moe, T, rows, cf, scale):
    """T * k / N rows an expert, whatever number of slots a token has."""
    cfg = dict(LAYER, routing=moe.MOE_ROUTING_EXPERT_CHOICE, capacity_factor=cf)
    T = T // scale
    assert moe.moe_capacity(cfg, T) == min(T, -(-T * scale * 8 // 128))
    assert moe.moe_expert_ffn_mx_tile_rows(cfg, T) == rows


def test_form_of_an_invalid_configuration(moe):
    assert moe.moe_expert_ffn_mx_tile_rows(dict(LAYER, hidden=100), 4) == 0
    assert moe.moe_expert_ffn_mx_tile_rows(LAYER, -1) == 0


@pytest.mark.parametrize("B", [8, 128])
def test_expert_choice_workspace_serves_fewer_tokens(moe, B):
    cfg = dict(LAYER, routing=moe.MOE_ROUTING_EXPERT_CHOICE, block_size=B)
    sizes = [moe.moe_workspace_bytes_mx(cfg, T) for T in range(0, 2000)]
    assert sizes == sorted(sizes)
