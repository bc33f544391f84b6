"""The 64-bit reference of the 4-bit expert path, and the refusals of its entry points (no GPU)."""
import ctypes

import numpy as np
import pytest

from tests import mx_ref
from tests.test_abi import moe  # noqa: F401  (the built library)

CFG = dict(hidden=256, num_experts=16, top_k=4, intermediate=128, block_size=8)


def test_grid_values_and_ties():
    row = np.zeros(32)
    row[:16] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -5.0, 5.01, 7.9, -7.9, 0.2501, 3.49]
    codes, scales = mx_ref.quantize(row[None])
    assert scales[0, 0] == 127
    got = mx_ref.dequantize(codes, scales)[0, :16]
    want = [6, 0, 1, 1, 2, 2, 4, 4, -0.0, -1, -4, 6, 6, -6, 0.5, 3]
    assert np.array_equal(got, want)


def test_scales_of_extreme_blocks():
    x = np.zeros((5, 32))
    x[1, 3] = 2.0 ** -133
    x[2, 3], x[3, 4], x[4, 5] = np.inf, np.nan, 3.3e38
    codes, scales = mx_ref.quantize(x)
    assert list(scales[:, 0]) == [0, 0, 255, 255, 127 + 125]
    v = mx_ref.dequantize(codes, scales)
    assert np.isnan(v[2:4]).all() and (v[:2] == 0).all() and v[4, 5] == 4 * 2.0 ** 126 - 2.0 ** 126


def test_requantizing_is_the_identity():
    rng = np.random.default_rng(0)
    v = mx_ref.dequantize(*mx_ref.quantize(rng.standard_normal((64, 96)) * 2.0 ** rng.integers(-20, 20, (64, 1))))
    assert np.array_equal(mx_ref.dequantize(*mx_ref.quantize(v)), v)


def test_route_ties_and_groups():
    l = np.zeros((1, 12))
    idx, gate, margin = mx_ref.route(l, None, 3, True, groups=4, top_groups=2, top2=True, renorm=True)
    assert list(idx[0]) == [0, 1, 2] and np.allclose(gate, 1 / 3) and margin[0] == 0
    l[0, 7], l[0, 8] = 2, 1
    idx, _, _ = mx_ref.route(l, None, 3, True, groups=4, top_groups=1)
    assert list(idx[0]) == [6, 7, 8]


def _call(moe, name, *args):
    return getattr(moe._lib, name)(*args)


OK16 = ctypes.c_void_p(1 << 20)      # an aligned address: refused calls never read it
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.mark.parametrize("bad,code", [
    (dict(score=2), 1), (dict(group_score=-1), 1), (dict(renormalize=2), 1), (dict(scale=float("nan")), 1),
    (dict(scale=-1.0), 1), (dict(num_groups=3), 1), (dict(num_groups=-1), 1), (dict(num_groups=4, top_groups=5), 1),
    (dict(num_groups=16, top_groups=4, group_score=1), 1),      # one expert a group has no second best
    (dict(num_groups=8, top_groups=1), 1)])                      # two experts left for four slots
def test_scoring_refusals(moe, bad, code):
    s = moe.make_scoring()
    for name, v in bad.items():
        setattr(s, name, v)
    assert moe.moe_check_scoring(CFG, s) == code


def test_scoring_accepts(moe):
    assert moe.moe_check_scoring(CFG, dict()) == 0
    assert moe.moe_check_scoring(CFG, dict(score=1, num_groups=8, top_groups=2, group_score=1, renormalize=True)) == 0
    assert moe.moe_check_scoring(dict(CFG, num_experts=64), dict(num_groups=64)) == 2
    assert moe.moe_check_scoring(dict(CFG, routing=1), dict()) == 1


def test_mx_refusals(moe):
    for K, code in ((0, 1), (33, 2), (16, 2), (-32, 1)):
        assert _call(moe, "moe_quantize_mx", 4, K, OK16, OK16, OK16, None) == code
        assert _call(moe, "moe_dequantize_mx", 4, K, OK16, OK16, OK16, None) == code
    assert _call(moe, "moe_quantize_mx", -1, 32, OK16, OK16, OK16, None) == 1
    assert _call(moe, "moe_quantize_mx", 1 << 40, 32, OK16, OK16, OK16, None) == 2
    assert _call(moe, "moe_quantize_mx", 0, 32, None, None, None, None) == 0
    for args in ((None, OK16, OK16), (OK16, ODD, OK16), (OK16, OK16, None)):
        assert _call(moe, "moe_quantize_mx", 4, 32, *args, None) == 1
        assert _call(moe, "moe_dequantize_mx", 4, 32, *args, None) == 1
        assert _call(moe, "moe_quantize_weights_mx", 2, 32, 8, *args, None) == 1
    assert _call(moe, "moe_quantize_weights_mx", 2, 32, 12, OK16, OK16, OK16, None) == 2
    assert _call(moe, "moe_quantize_weights_mx", 2, 48, 8, OK16, OK16, OK16, None) == 2
    assert _call(moe, "moe_quantize_weights_mx", -2, 32, 8, OK16, OK16, OK16, None) == 1
    assert _call(moe, "moe_pack_scales_mx", 2, 64, 128, 0, OK16, OK16, None) == 2
    assert _call(moe, "moe_pack_scales_mx", 2, 128, 96, 0, OK16, OK16, None) == 2
    assert _call(moe, "moe_pack_scales_mx", 2, 128, 128, 2, OK16, OK16, None) == 1
    assert _call(moe, "moe_pack_scales_mx", 2, 128, 128, 0, OK16, ODD, None) == 1


def test_norm_refusals(moe):
    def call(T=2, H=64, x=OK16, r=OK16, w=OK16, eps=1e-6, ro=OK16, out=OK16, c=OK16, s=OK16):
        return moe._lib.moe_add_norm(T, H, x, r, w, eps, ro, out, c, s, None)
    assert call(T=0) == 0 and call(T=0, x=None) == 0
    for bad, code in ((dict(T=-1), 1), (dict(H=0), 1), (dict(H=48), 2), (dict(H=65536), 2), (dict(eps=-1.0), 1),
                      (dict(eps=float("nan")), 1), (dict(x=None), 1), (dict(w=ODD), 1), (dict(r=ODD), 1),
                      (dict(c=None), 1), (dict(s=None), 1), (dict(out=None, c=None, s=None), 1)):
        assert call(**bad) == code, bad


def test_ffn_refusals(moe):
    cfg = moe.make_config(**CFG)
    n = moe.moe_workspace_bytes_mx(cfg, 8)
    assert n > 0 and moe.moe_workspace_bytes_mx(dict(CFG, hidden=100), 8) == 0
    for c in (CFG, dict(CFG, num_experts=128, top_k=8, block_size=16), dict(CFG, num_experts=1, top_k=1)):
        sizes = [moe.moe_workspace_bytes_mx(c, T) for T in range(0, 1200)]   # across every tile height
        assert sizes == sorted(sizes)

    def call(c=cfg, T=8, at=None, value=None, ws_bytes=n):
        ptrs = [OK16] * 6 + [None] * 4 + [OK16] * 4 + [None, OK16]
        if at is not None:
            ptrs[at] = value
        return moe._lib.moe_expert_ffn_mx(ctypes.byref(c), T, *ptrs, ws_bytes, None)
    assert call(T=0) == 0
    assert call(T=-1) == 1
    assert call(ws_bytes=n - 1) == 3
    for at in (*range(6), *range(10, 14), 15):
        assert call(at=at) == 1 and call(at=at, value=ODD) == 1
    shared = moe.make_config(**dict(CFG, shared_intermediate=128))
    assert call(c=shared, ws_bytes=1 << 40) == 1           # the shared expert's weights are missing
    assert call(c=moe.make_config(**dict(CFG, hidden=96))) == 2


def test_forward_refusals(moe):
    cfg, sc = moe.make_config(**CFG), moe.make_scoring()
    n = moe.moe_workspace_bytes_mx(cfg, 8)

    def call(c=cfg, s=sc, T=8, eps=1e-6, at=None, ws_bytes=n):
        p = [OK16, None, OK16, OK16, None, None, OK16, OK16, OK16, OK16, None, None, None, None, OK16, OK16]
        if at is not None:
            p[at] = ODD
        return moe._lib.moe_forward_mx(ctypes.byref(c), ctypes.byref(s), T, *p[:3], eps, *p[3:], ws_bytes, None)
    assert call(T=0) == 0 and call(T=-1) == 1 and call(eps=-1.0) == 1 and call(ws_bytes=n - 1) == 3
    for at in (*range(10), 14, 15):
        assert call(at=at) == 1, at
    assert call(s=moe.make_scoring(num_groups=3)) == 1
    assert call(c=moe.make_config(**dict(CFG, capacity_factor=1.0, overflow_policy=1))) == 1


def test_python_checks(moe):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_quantize_mx(x, c, s)
    with pytest.raises(ValueError, match="x:"):
        moe.moe_quantize_mx(x.float(), c, s)
    with pytest.raises(ValueError, match="logits"):
        moe.moe_route_scored(CFG, dict(), torch.zeros(4, 15), None, None, None)
    with pytest.raises(ValueError, match="weight"):
        moe._want("weight", torch.zeros(8, 8).t(), "float32", (8, 8))
