"""Outputs of the training step's entry points that lie over an input, the workspace or another output are refused
before any launch (no GPU needed)."""
import ctypes

import pytest

from tests.test_abi import moe  # noqa: F401

T, H, I, N, S, B, K, F = 64, 128, 256, 8, 2, 8, 128, 512
ROWS = T * S + N * (B - 1)
CFG = dict(hidden=H, num_experts=N, top_k=S, intermediate=I, block_size=B)
INVALID = 1
# addresses far enough apart for every tensor of these sizes
(GU, GATE, DA, IDS, PADDED, DGU, DGATE, A, X, R, W, BIAS, OUT, V, DOUT, DX, DW, DB, WS, COUNTS, Y) = (
    0x100000000 * i for i in range(1, 22))


def over(start, size, n):
    """Addresses of n bytes that share 16 with [start, start + size): at its start, at its end, and (n larger) from before it."""
    return [start, start + size - 16] + ([start - n + 16] if start >= n else [])


def swiglu(moe, **kw):  # noqa: F811
    t = dict(dict(gu=GU, gate=GATE, ids=IDS, padded=PADDED, a=A), **kw)
    return moe._lib.moe_swiglu(ctypes.byref(moe.make_config(**CFG)), T, t["gu"], t["gate"], t["ids"], t["padded"], t["a"],
                               None)


def swiglu_backward(moe, **kw):  # noqa: F811
    t = dict(dict(gu=GU, gate=GATE, da=DA, ids=IDS, padded=PADDED, dgu=DGU, dgate=DGATE, a=A), **kw)
    return moe._lib.moe_swiglu_backward(ctypes.byref(moe.make_config(**CFG)), T, t["gu"], t["gate"], t["da"], t["ids"],
                                        t["padded"], t["dgu"], t["dgate"], t["a"], None)


SWIGLU = dict(gu=(GU, ROWS * 2 * I * 2), gate=(GATE, T * S * 4), da=(DA, ROWS * I * 2), ids=(IDS, ROWS * 4),
              padded=(PADDED, 16), dgu=(DGU, ROWS * 2 * I * 2), dgate=(DGATE, T * S * 4), a=(A, ROWS * I * 2))


@pytest.mark.parametrize("under", ["gu", "gate", "ids", "padded"])
def test_swiglu(moe, under):  # noqa: F811
    for p in over(*SWIGLU[under], SWIGLU["a"][1]):
        assert swiglu(moe, a=p) == INVALID


@pytest.mark.parametrize("out,under", [(o, u) for o in ("dgu", "dgate", "a") for u in SWIGLU if u != o])
def test_swiglu_backward(moe, out, under):  # noqa: F811
    in_place = {("dgu", "gu"), ("a", "da")}
    for p in over(*SWIGLU[under], SWIGLU[out][1]):
        if (out, under) not in in_place or p != SWIGLU[under][0]:
            assert swiglu_backward(moe, **{out: p}) == INVALID


@pytest.mark.parametrize("out,under", [("dgate", "gu"), ("dgate", "da"), ("dgate", "ids")])
def test_swiglu_backward_in_place(moe, out, under):  # noqa: F811
    """What is in place of an input is an output all the same."""
    for p in over(*SWIGLU[under], SWIGLU[out][1]):
        assert swiglu_backward(moe, dgu=GU, a=DA, **{out: p}) == INVALID


def layer_norm(moe, **kw):  # noqa: F811
    t = dict(dict(x=X, r=R, w=W, b=BIAS, ro=V, out=OUT), **kw)
    return moe._lib.moe_add_layer_norm(T, H, t["x"], t["r"], t["w"], t["b"], 1e-5, t["ro"], t["out"], None)


NORM = dict(x=(X, T * H * 2), r=(R, T * H * 2), w=(W, H * 2), b=(BIAS, H * 2), ro=(V, T * H * 2), out=(OUT, T * H * 2))


@pytest.mark.parametrize("out,under", [(o, u) for o in ("ro", "out") for u in NORM if u != o])
def test_add_layer_norm(moe, out, under):  # noqa: F811
    for p in over(*NORM[under], NORM[out][1]):
        if under not in ("x", "r") or p != NORM[under][0]:   # in place
            assert layer_norm(moe, **{out: p}) == INVALID


def norm_backward(moe, n, **kw):  # noqa: F811
    t = dict(dict(v=V, dout=DOUT, r=R, w=W, dx=DX, dw=DW, db=DB, ws=WS), **kw)
    return moe._lib.moe_norm_backward(T, H, 1, t["v"], t["dout"], t["r"], t["w"], 1e-5, t["dx"], t["dw"], t["db"], t["ws"],
                                      n, None)


@pytest.mark.parametrize("out", ["dx", "dw", "db", "ws"])
@pytest.mark.parametrize("under", ["v", "dout", "r", "w", "dx", "dw", "db", "ws"])
def test_norm_backward(moe, out, under):  # noqa: F811
    if out == under:
        return
    n = moe.moe_workspace_bytes_norm_backward(T, H)
    at = dict(v=(V, T * H * 2), dout=(DOUT, T * H * 2), r=(R, T * H * 2), w=(W, H * 2), dx=(DX, T * H * 2), dw=(DW, H * 4),
              db=(DB, H * 4), ws=(WS, n))
    for p in over(*at[under], at[out][1]):
        if (out, under) != ("dx", "r") or p != R:   # in place
            assert norm_backward(moe, n, **{out: p}) == INVALID


def grouped(moe, op, **kw):  # noqa: F811
    c = moe.make_config(**CFG)
    t = dict(dict(x=X, w=W, dy=DOUT, ids=IDS, counts=COUNTS, y=Y, dw=DW, add=None, ws=WS), **kw)
    if op == "gemm":
        return moe._lib.moe_grouped_gemm(ctypes.byref(c), T, K, F, 1, t["x"], t["w"], t["ids"], t["counts"], t["y"],
                                         t["ws"], 256, None)
    return moe._lib.moe_grouped_wgrad(ctypes.byref(c), T, K, F, 1, t["x"], t["dy"], t["ids"], t["counts"], t["add"],
                                      t["dw"], t["ws"], 256, None)


GROUPED = dict(x=(X, T * K * 2), w=(W, N * K * F * 2), dy=(DOUT, ROWS * F * 2), ids=(IDS, ROWS * 4), counts=(COUNTS, N * 4),
               ws=(WS, 256), y=(Y, ROWS * F * 2), dw=(DW, N * K * F * 4), add=(GU, N * K * F * 4))


@pytest.mark.parametrize("op,out,under", [("gemm", o, u) for o in ("y", "ws") for u in ("x", "w", "ids", "counts", "ws", "y")
                                          if u != o] +
                         [("wgrad", o, u) for o in ("dw", "ws") for u in ("x", "dy", "ids", "counts", "add", "ws", "dw")
                          if u != o])
def test_grouped(moe, op, out, under):  # noqa: F811
    for p in over(*GROUPED[under], GROUPED[out][1]):
        if (out, under) != ("dw", "add") or p != GU:   # in place
            assert grouped(moe, op, **{out: p}, **({"add": GU} if op == "wgrad" else {})) == INVALID
