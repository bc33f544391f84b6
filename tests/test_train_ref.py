"""The 64-bit formulas of the training step's tests against central differences."""
import pytest
import torch

from tests import train_ref as R


def _numeric(f, x, h=1e-6):
    """Gradient of the scalar f by central differences."""
    g = torch.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.numel()):
        v = flat[i].item()
        flat[i] = v + h
        up = f()
        flat[i] = v - h
        out[i] = (up - f()) / (2 * h)
        flat[i] = v
    return g


def _randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=R.F64)


def test_swiglu_backward():
    g, u, w, da = 2 * _randn(3, 8), _randn(3, 8, seed=1), _randn(3, 1, seed=2), _randn(3, 8, seed=3)

    def f():
        return (R.swiglu(g, u, w) * da).sum()
    dg, du, dw = R.swiglu_backward(g, u, w, da)
    for x, d in ((g, dg), (u, du), (w, dw.unsqueeze(-1))):
        assert torch.allclose(_numeric(f, x), d, atol=1e-7)


@pytest.mark.parametrize("centre", [True, False])
def test_norm_backward(centre):
    v, dout, dres = 1 + _randn(4, 16), _randn(4, 16, seed=1), _randn(4, 16, seed=2)
    w, b = 1 + 0.2 * _randn(16, seed=3), _randn(16, seed=4)

    def f():
        out = R.layer_norm(v, w, b, 1e-5) if centre else R.rms_norm(v, w, 1e-5)
        return (out * dout).sum() + (v * dres).sum()
    dx, dw, db, *_ = R.norm_backward(v, dout, dres, w, 1e-5, centre)
    for x, d in ((v, dx), (w, dw)) + (((b, db),) if centre else ()):
        assert torch.allclose(_numeric(f, x), d, atol=1e-7)


@pytest.mark.parametrize("gather,transposed", [(False, False), (True, False), (False, True), (True, True)])
def test_grouped_products(gather, transposed):
    G = R.Groups(5, 4, 2, 8, device="cpu", idle=(1,))
    assert G.counts[1] == 0 and sum(G.counts) == 10
    K, F = 8, 16
    g = torch.Generator().manual_seed(5)
    x = torch.randn(5, K, generator=g, dtype=R.F64) if gather else G.grouped(K, g, fill=0.0).double()
    w = _randn(4, F, K) if transposed else _randn(4, K, F)
    dy = G.grouped(F, g, fill=0.0).double()

    def f():
        return (R.gemm(G, x, w, gather, transposed)[0] * dy).sum()
    dw, _ = R.wgrad(G, x, dy, gather, False)
    assert torch.allclose(_numeric(f, w), dw.transpose(1, 2) if transposed else dw, atol=1e-7)
    # the input's gradient is the product with the other form of the same weights
    dx, _ = R.gemm(G, dy, w, False, not transposed)
    if gather:   # a token sums its rows
        sums = torch.zeros(5, K, dtype=R.F64)
        sums.index_add_(0, torch.cat([G.token(p, n) for p, n in zip(G.start, G.counts)]), dx[G.real])
        dx = sums
    assert torch.allclose(_numeric(f, x), dx, atol=1e-7)
