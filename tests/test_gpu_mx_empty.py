"""The 4-bit FFN on a list without a row (every route dropped elsewhere): nothing is written, the shared expert runs."""
import numpy as np
import pytest

from tests import mx_ref
from tests.test_gpu_mx import Layer, _tokens, f64, moe, torch_  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,form", [(3, 32), (80, 128), (500, 256)])
@pytest.mark.parametrize("Is", [0, 128])
def test_empty_list(moe, T, form, Is):
    torch = torch_()
    L = Layer(moe, 256, 4, 1, 128, 16, Is, seed=T)
    assert moe.moe_expert_ffn_mx_tile_rows(L.cfg, T) == form
    c, s = _tokens(np.random.default_rng(T), T, 256)
    e = dict(device="cuda", dtype=torch.int32)
    d = dict(ids=torch.full((moe.moe_max_padded_rows(L.cfg, T),), -1, **e),
             blocks=torch.full((moe.moe_max_blocks(L.cfg, T),), -1, **e), npad=torch.zeros(1, **e))
    y, ysh = L.ffn(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), d)
    assert (y == 7.0).all()
    if Is:
        ref, tol = mx_ref.ffn_rows(mx_ref.dequantize(c, s), L.val[2][0], L.val[3][0])
        assert (np.abs(f64(ysh) - ref) <= tol).all()
