"""Argument checks of the training step's entry points: they return before any launch (no GPU needed)."""
import ctypes

import pytest

from tests.test_abi import moe  # noqa: F401

CFG = dict(hidden=128, num_experts=8, top_k=2, intermediate=256, block_size=8)
WS = 256
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
# addresses far enough apart for every tensor of these sizes
X, W, IDS, COUNTS, Y, WSP = (0x100000000 * i for i in range(1, 7))


def gemm(moe, cfg=CFG, T=64, K=128, F=512, flags=1, x=X, w=W, ids=IDS, counts=COUNTS, y=Y, ws=WSP, n=WS):
    c = moe.make_config(**cfg)
    return moe._lib.moe_grouped_gemm(ctypes.byref(c), T, K, F, flags, x, w, ids, counts, y, ws, n, None)


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), INVALID), (dict(T=1 << 21), UNSUPPORTED), (dict(K=0), INVALID), (dict(F=-8), INVALID),
    (dict(K=12), UNSUPPORTED), (dict(F=65544), UNSUPPORTED), (dict(flags=4), INVALID), (dict(x=None), INVALID),
    (dict(x=X + 8), INVALID), (dict(w=None), INVALID), (dict(ids=None), INVALID), (dict(flags=0, ids=IDS + 4), INVALID),
    (dict(counts=None), INVALID), (dict(y=None), INVALID), (dict(ws=None), INVALID), (dict(n=WS - 1), WORKSPACE),
    (dict(y=X), INVALID), (dict(y=X + 64 * 128 * 2 - 16), INVALID), (dict(y=W + 8 * 128 * 512 * 2 - 16), INVALID),
    (dict(cfg=dict(CFG, hidden=100)), UNSUPPORTED), (dict(cfg=dict(CFG, block_size=12)), UNSUPPORTED)])
def test_grouped_gemm(moe, bad, code):
    assert gemm(moe, **bad) == code


def wgrad(moe, cfg=CFG, T=64, K=128, F=512, flags=1, x=X, dy=W, ids=IDS, counts=COUNTS, add=None, dw=Y, ws=WSP, n=WS):
    c = moe.make_config(**cfg)
    return moe._lib.moe_grouped_wgrad(ctypes.byref(c), T, K, F, flags, x, dy, ids, counts, add, dw, ws, n, None)


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), INVALID), (dict(K=4), UNSUPPORTED), (dict(F=0), INVALID), (dict(flags=8), INVALID),
    (dict(flags=4, add=0x900000000), INVALID), (dict(add=0x900000008), INVALID), (dict(add=Y + 16), INVALID),
    (dict(x=None), INVALID), (dict(dy=None), INVALID), (dict(ids=None), INVALID), (dict(flags=2, ids=None), INVALID),
    (dict(counts=None), INVALID), (dict(dw=None), INVALID), (dict(ws=WSP + 4), INVALID), (dict(n=0), WORKSPACE),
    (dict(dw=X), INVALID), (dict(dw=W), INVALID)])
def test_grouped_wgrad(moe, bad, code):
    assert wgrad(moe, **bad) == code


def test_no_tokens(moe):
    assert gemm(moe, T=0, x=None, w=None, ids=None, counts=None, y=None, ws=None, n=0) == 0
    assert wgrad(moe, T=0, x=None, dy=None, ids=None, counts=None, add=Y, ws=None, n=0) == 0   # dw_add is dw
    assert wgrad(moe, T=0, dw=None) == INVALID
    c = moe.make_config(**CFG)
    assert moe._lib.moe_swiglu(ctypes.byref(c), 0, *[None] * 6) == 0
    assert moe._lib.moe_swiglu_backward(ctypes.byref(c), 0, *[None] * 9) == 0
    assert moe._lib.moe_add_layer_norm(0, 128, *[None] * 4, 1e-5, *[None] * 3) == 0
    assert moe._lib.moe_norm_backward(0, 128, 1, *[None] * 4, 1e-5, *[None] * 4, 0, None) == 0


A, DA, DGU, DG = (0x100000000 * i for i in range(11, 15))


@pytest.mark.parametrize("i,value", [(0, None), (0, X + 2), (1, W + 4), (2, None), (3, None), (4, None),
                                     (4, X), (4, X + 2 * 128 * 256 * 2)])
def test_swiglu(moe, i, value):
    args = [X, W, IDS, COUNTS, A]
    args[i] = value
    c = moe.make_config(**CFG)
    assert moe._lib.moe_swiglu(ctypes.byref(c), 64, *args, None) == INVALID


@pytest.mark.parametrize("i,value", [(0, None), (2, None), (3, None), (4, None), (5, None), (5, X + 16), (5, DA), (6, DG + 4),
                                     (7, X), (7, DGU), (7, DA + 16)])
def test_swiglu_backward(moe, i, value):
    args = [X, W, DA, IDS, COUNTS, DGU, DG, A]
    args[i] = value
    c = moe.make_config(**CFG)
    assert moe._lib.moe_swiglu_backward(ctypes.byref(c), 64, *args, None) == INVALID


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=12), UNSUPPORTED), (dict(H=32776), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(x=None), INVALID), (dict(r=X + 2), INVALID),
    (dict(w=None), INVALID), (dict(b=COUNTS + 8), INVALID), (dict(out=None), INVALID), (dict(out=X + 16), INVALID),
    (dict(ro=Y), INVALID), (dict(ro=X, out=X), INVALID)])
def test_add_layer_norm(moe, bad, code):
    a = dict(dict(T=4, H=128, x=X, r=W, w=IDS, b=COUNTS, eps=1e-5, ro=A, out=Y), **bad)
    assert moe._lib.moe_add_layer_norm(a["T"], a["H"], a["x"], a["r"], a["w"], a["b"], a["eps"], a["ro"], a["out"],
                                       None) == code


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), INVALID), (dict(H=4), UNSUPPORTED), (dict(centre=2), INVALID), (dict(eps=-1.0), INVALID),
    (dict(v=None), INVALID), (dict(dout=None), INVALID), (dict(dres=A + 2), INVALID), (dict(w=None), INVALID),
    (dict(dx=None), INVALID), (dict(dx=X), INVALID), (dict(dx=W + 16), INVALID), (dict(dx=A + 16), INVALID),
    (dict(dw=DA + 8), INVALID), (dict(ws=None), INVALID), (dict(n=-1), WORKSPACE)])
def test_norm_backward(moe, bad, code):
    a = dict(dict(T=4, H=128, centre=1, v=X, dout=W, dres=A, w=IDS, eps=1e-5, dx=Y, dw=DA, db=DG, ws=WSP, n=0), **bad)
    n = moe.moe_workspace_bytes_norm_backward(4, 128) + a["n"]
    assert n > 0
    assert moe._lib.moe_norm_backward(a["T"], a["H"], a["centre"], a["v"], a["dout"], a["dres"], a["w"], a["eps"],
                                      a["dx"], a["dw"], a["db"], a["ws"], n, None) == code


def test_workspaces(moe):
    assert moe.moe_workspace_bytes_grouped(CFG, 64) == WS
    assert moe.moe_workspace_bytes_grouped(dict(CFG, hidden=100), 64) == 0
    assert moe.moe_workspace_bytes_grouped(CFG, -1) == 0
    sizes = [moe.moe_workspace_bytes_norm_backward(T, 4096) for T in (1, 64, 16448)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert moe.moe_workspace_bytes_norm_backward(64, 100) == 0


def test_binding_checks_tensors(moe):
    import torch
    x = torch.zeros(64, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x: a contiguous CUDA tensor"):
        moe.moe_grouped_gemm(CFG, 64, x, x, None, None, x, None, gather=True)
    with pytest.raises(ValueError, match="x: a 2-D tensor"):
        moe.moe_grouped_wgrad(CFG, 64, None, x, None, None, x, None)
    with pytest.raises(ValueError, match="gu"):
        moe.moe_swiglu(CFG, 64, x, None, None, None, x)
    with pytest.raises(ValueError, match="x"):
        moe.moe_add_layer_norm(x, None, x, None, 1e-5, None, x)
    with pytest.raises(ValueError, match="v"):
        moe.moe_norm_backward(x, x, None, x, 1e-5, x, None, None, None)


def test_binding_refuses_another_device(moe, monkeypatch):
    class Elsewhere:
        device = "cuda:1"

        def get_device(self):
            return 1
    monkeypatch.setattr(moe, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="x: on cuda:1, but the current device is cuda:0"):
        moe._here("x", Elsewhere())
    monkeypatch.setattr(moe, "_current_device", lambda: 1)
    moe._here("x", Elsewhere())


def test_rows_of_the_binding_and_the_library(moe):
    for kw in (dict(), dict(capacity_factor=1.5), dict(routing=1), dict(routing=1, capacity_factor=0.3)):
        for T in (0, 1, 7, 1000):
            c = moe.make_config(**CFG, **kw)
            assert moe._rows(c, T) == moe.moe_max_padded_rows(c, T)


@pytest.mark.parametrize("dw,db", [(DA, DA), (DA, DA + 128 * 4 - 16), (Y + 16, DG), (DA, Y), (WSP, DG), (None, WSP)])
def test_norm_backward_refuses_sums_over_one_another(moe, dw, db):
    n = moe.moe_workspace_bytes_norm_backward(4, 128)
    assert moe._lib.moe_norm_backward(4, 128, 1, X, W, A, IDS, 1e-5, Y, dw, db, WSP, n, None) == INVALID


@pytest.mark.parametrize("dgate", [W, W + 64 * 2 * 4 - 16, DGU + 16, A])
def test_swiglu_backward_refuses_gates_over_other_tensors(moe, dgate):
    c = moe.make_config(**CFG)
    assert moe._lib.moe_swiglu_backward(ctypes.byref(c), 64, X, W, DA, IDS, COUNTS, DGU, dgate, A, None) == INVALID
