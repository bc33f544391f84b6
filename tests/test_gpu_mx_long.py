"""The 4-bit FFN over reductions of more steps than its pipelines have stages, and its workspace shared by calls of
every size."""
import numpy as np
import pytest

from tests import mx_ref
from tests.gpu_util import host
from tests.test_gpu_mx import Layer, _check_rows, _tokens, moe, torch_  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", params=[(4224, 5120), (5376, 4480)], ids=str)
def layer(moe, request):  # noqa: F811
    """33 and 40, 42 and 35 chunks of 128 elements: an odd and an even number in each product."""
    H, I = request.param
    return Layer(moe, H, 3, 1, I, 8, seed=I)


@pytest.mark.parametrize("T,form,rows", [(10, 32, None), (140, 128, None), (400, 256, 60)])
def test_long_reductions(moe, layer, T, form, rows):
    """Against the 64-bit reference: stages and scale slots are used again within one sum."""
    torch = torch_()
    L, H = layer, layer.H
    assert moe.moe_expert_ffn_mx_tile_rows(L.cfg, T) == form
    rng = np.random.default_rng(H + T)
    c, s = _tokens(rng, T, H)
    idx = np.where(rng.random(T) < 0.8, 1, 2).astype(np.int32).reshape(T, 1)
    d = L.dispatch(torch.from_numpy(idx).cuda())
    y, _ = L.ffn(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), d)
    routed = np.flatnonzero(host(d["ids"])[:int(d["npad"][0])] < T)
    some = None if rows is None else rng.choice(routed, rows, replace=False)
    _check_rows(L, y, mx_ref.dequantize(c, s), d, some)


@pytest.mark.parametrize("N,k,B,Is", [(16, 2, 8, 128), (4, 2, 128, 0)])
def test_one_workspace_serves_every_size(moe, N, k, B, Is):
    """Calls of every form in a workspace made for the largest, filled with other bytes first: the bits of a workspace
    of their own."""
    torch = torch_()
    L = Layer(moe, 256, N, k, 384, B, Is, seed=N)
    rng = np.random.default_rng(N)
    big = moe.workspace_mx(L.cfg, 2000)
    big.fill_(0xFF)
    x, xs = (torch.from_numpy(v).cuda() for v in _tokens(rng, 2000, 256))
    idx = torch.from_numpy(np.sort(np.argsort(rng.random((2000, N)), axis=1)[:, :k], axis=1).astype(np.int32)).cuda()
    forms = set()
    for T in (2000, 1, 700, 40, 129, 8, 1999, 300):
        forms.add(moe.moe_expert_ffn_mx_tile_rows(L.cfg, T))
        d = L.dispatch(idx[:T].contiguous())
        c, s = x[:T].contiguous(), xs[:T].contiguous()
        own = torch.full((moe.moe_workspace_bytes_mx(L.cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")
        want, want_sh = L.ffn(c, s, d, own)
        y, ysh = L.ffn(c, s, d, big)
        assert torch.equal(y, want) and (ysh is None or torch.equal(ysh, want_sh)), T
    assert forms == {32, 128, 256}
