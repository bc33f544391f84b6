"""The 4-bit expert FFN on an expert-choice layout (a slot for every expert) against its 64-bit reference."""
import numpy as np
import pytest

from tests import mx_ref
from tests.gpu_util import host
from tests.test_gpu_mx import Layer, _check_rows, _tokens, moe, torch_  # noqa: F401

pytestmark = pytest.mark.gpu


def _layout(moe, L, T, rng):
    torch = torch_()
    logits = torch.from_numpy(rng.standard_normal((T, L.N)).astype(np.float32)).cuda()
    rows, R = moe.moe_max_padded_rows(L.cfg, T), T * L.N
    e = dict(device="cuda", dtype=torch.int32)
    d = dict(ids=torch.full((rows,), -9, **e), blocks=torch.full((moe.moe_max_blocks(L.cfg, T),), -9, **e),
             npad=torch.zeros(1, **e), pos=torch.empty(R, **e))
    moe.moe_route_expert_choice(L.cfg, logits, torch.empty(R, device="cuda"), torch.empty(R, dtype=torch.uint8, device="cuda"),
                                d["pos"], d["ids"], d["blocks"], d["npad"], torch.empty(L.N, **e), moe.workspace(L.cfg, T))
    return d


@pytest.mark.parametrize("T,B,cf,form", [
    (1, 8, 0.0, 32),         # each expert takes the one token
    (64, 8, 0.0, 32),
    (100, 128, 0.0, 32),     # tiles shorter than a block
    (256, 16, 0.0, 128),
    (255, 128, 1.5, 128),
    (1024, 32, 0.0, 256),
    (300, 8, 100.0, 256)])   # every token to every expert
def test_expert_choice(moe, T, B, cf, form):
    torch = torch_()
    L = Layer(moe, 256, 16, 2, 384, B, Is=128, seed=T, routing=1, capacity_factor=cf)
    L.k = L.N                # slots a token
    assert moe.moe_expert_ffn_mx_tile_rows(L.cfg, T) == form
    rng = np.random.default_rng(T)
    c, s = _tokens(rng, T, 256)
    d = _layout(moe, L, T, rng)
    y, ysh = L.ffn(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), d)
    xv = mx_ref.dequantize(c, s)
    assert int((host(d["ids"])[:int(d["npad"][0])] < T * L.N).sum()) == L.N * moe.moe_capacity(L.cfg, T)
    _check_rows(L, y, xv, d)
    ref, tol = mx_ref.ffn_rows(xv, L.val[2][0], L.val[3][0])
    assert (np.abs(ysh.float().cpu().numpy() - ref) <= tol).all()
