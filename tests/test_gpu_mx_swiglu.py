"""SwiGLU of the 4-bit FFN with gates far from zero: blocks whose values are all tiny, or all about |g * u|."""
import numpy as np
import pytest

from tests import mx_ref
from tests.test_gpu_mx import Layer, _tokens, f64, moe, torch_  # noqa: F401

pytestmark = pytest.mark.gpu


def _rows(x, w13, w2):
    """y in 64 bits and its bound: the pre-activation's sums, the exponent's rounded product (max(-g, 0) 2^-23 of silu,
    both ends of its interval), 2^-20 for the rest, the 4-bit rounding of an interval, W2's sums and bf16."""
    H, I = x.shape[1], w2.shape[1]
    gu = x @ w13.T
    err = (H / 64 + 64) * 2.0 ** -23 * (np.abs(x) @ np.abs(w13).T)
    g, u, eg, eu = gu[:, :I], gu[:, I:], err[:, :I], err[:, I:]
    silu = g / (1.0 + np.exp(-g))
    a = silu * u
    rel = 2.0 ** -20 + np.maximum(eg - g, 0.0) * 2.0 ** -23
    # silu over g +- eg: its derivative is at most max(1.1, (1 + |g|) sigmoid) in size
    slope = np.where(g < -2, (1.0 + np.abs(g)) * np.exp(np.minimum(g + eg, 0.0)), 1.1)
    ds = slope * eg + rel * np.abs(silu)
    lo, hi = mx_ref._mx_interval(a, ds * (np.abs(u) + eu) + np.abs(silu) * eu)
    q = mx_ref.dequantize(*mx_ref.quantize(a))
    y = q @ w2.T
    tol = np.maximum(hi - q, q - lo) @ np.abs(w2).T + (I / 64 + 64) * 2.0 ** -23 * (np.abs(q) @ np.abs(w2).T)
    return g, y, tol * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(y)


@pytest.mark.parametrize("T", [5, 120, 300])   # swapped, single CTAs, CTA pairs
@pytest.mark.parametrize("gate", [-70.0, -40.0, -12.0, 40.0])
def test_gates_far_from_zero(moe, T, gate):
    torch = torch_()
    H, I, N = 256, 256, 2
    L = Layer(moe, H, N, 1, I, 8, seed=T)
    rng = np.random.default_rng(T)
    x = np.abs(rng.standard_normal((T, H))) + 0.5
    c, s = mx_ref.quantize(x)
    xv = mx_ref.dequantize(c, s)
    w13 = rng.standard_normal((N, 2 * I, H)) * 0.05
    w13[:, :I] = gate / xv.sum(1).mean() * (1 + 0.2 * rng.standard_normal((N, I, H)))   # every gate near `gate`
    cw, sw = mx_ref.quantize(w13)
    L.val[0] = mx_ref.dequantize(cw, sw)
    sd = torch.from_numpy(sw).cuda()
    L.dev[0], L.dev[1] = torch.from_numpy(cw).cuda(), torch.empty_like(sd)
    moe.moe_pack_scales_mx(sd, L.dev[1], True)
    idx = torch.from_numpy((np.arange(T) % N).astype(np.int32)).cuda().reshape(T, 1)
    d = L.dispatch(idx)
    y, _ = L.ffn(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), d)
    got = f64(y)[d["pos"].cpu().numpy()]
    for e in range(N):
        at = np.arange(e, T, N)
        g, ref, tol = _rows(xv[at], L.val[0][e], L.val[1][e])
        assert (np.sign(g) == np.sign(gate)).all() and np.abs(g).mean() > 0.7 * abs(gate)
        assert np.abs(ref).max() > 0
        assert (np.abs(got[at] - ref) <= tol).all(), float((np.abs(got[at] - ref) / tol).max())
        assert np.median(tol / np.abs(ref).clip(1e-300)) < 1.0   # the bound says something
