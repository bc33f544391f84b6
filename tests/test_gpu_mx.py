"""The 4-bit expert path on the GPU against its 64-bit reference."""
import numpy as np
import pytest

from tests import mx_ref
from tests.gpu_util import host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import invariant_expert_routing_gb300 as m
    return m


def torch_():
    import torch
    return torch


def bf16(a):
    """fp values (numpy) to a bf16 CUDA tensor."""
    torch = torch_()
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().bfloat16()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def mx_buffers(lead, K):
    torch = torch_()
    return (torch.full((*lead, K // 2), 0xAA, dtype=torch.uint8, device="cuda"),
            torch.full((*lead, K // 32), 0xAA, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------ conversion
def _awkward(rng, rows, K):
    x = rng.standard_normal((rows, K)).astype(np.float32)
    x *= (2.0 ** rng.integers(-126, 120, (rows, K // 32)).astype(np.float64)).repeat(32, 1).astype(np.float32)
    flat = x.reshape(-1, 32)
    flat[0] = 0
    if len(flat) > 8:
        flat[1] = np.tile([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -5, 7.9, -7.9, 0, -0.0, 4], 2)
        flat[2, 5], flat[3, 31], flat[4, 0] = np.inf, np.nan, -np.inf
        flat[5] = 0
        flat[5, 7] = 2.0 ** -133                      # the smallest bf16
        flat[6, 9] = 3.3895314e38                     # the largest
        flat[7] = -0.0
    return x


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 32), (1, 96), (7, 160), (37, 2048), (1025, 352), (2, 32768)])
def test_quantize_rows(moe, rows, K):
    x = bf16(_awkward(np.random.default_rng(rows * K), rows, K))
    codes, scales = mx_buffers((rows,), K)
    moe.moe_quantize_mx(x, codes, scales)
    rc, rs = mx_ref.quantize(f64(x))
    np.testing.assert_array_equal(host(scales), rs)
    np.testing.assert_array_equal(host(codes), rc)
    out = torch_().empty_like(x)
    moe.moe_dequantize_mx(codes, scales, out)
    np.testing.assert_array_equal(f64(out), mx_ref.dequantize(rc, rs))


def test_dequantize_every_scale(moe):
    torch = torch_()
    codes = torch.arange(256, device="cuda").to(torch.uint8).repeat(16).reshape(256, 16).contiguous()
    scales = torch.arange(256, device="cuda").to(torch.uint8).reshape(256, 1).contiguous()
    out = torch.empty(256, 32, dtype=torch.bfloat16, device="cuda")
    moe.moe_dequantize_mx(codes, scales, out)
    want = torch.from_numpy(mx_ref.dequantize(host(codes), host(scales))).bfloat16()
    np.testing.assert_array_equal(f64(out), f64(want))


@pytest.mark.parametrize("E,K,F", [(1, 32, 8), (3, 96, 40), (2, 288, 72), (2, 512, 136)])
def test_quantize_weights(moe, E, K, F):
    x = _awkward(np.random.default_rng(E * K * F), E * F, K).reshape(E, F, K)
    w = bf16(x.transpose(0, 2, 1))
    codes, scales = mx_buffers((E, F), K)
    moe.moe_quantize_weights_mx(w, codes, scales)
    rc, rs = mx_ref.quantize(f64(w).transpose(0, 2, 1))
    np.testing.assert_array_equal(host(scales), rs)
    np.testing.assert_array_equal(host(codes), rc)


@pytest.mark.parametrize("gate_up", [False, True])
def test_pack_scales_keeps_every_byte(moe, gate_up):
    torch = torch_()
    E, rows, K = 3, 256, 384
    s = torch.from_numpy(np.random.default_rng(1).integers(0, 256, (E, rows, K // 32), dtype=np.uint8)).cuda()
    packed = torch.empty_like(s)
    moe.moe_pack_scales_mx(s, packed, gate_up)
    order = np.arange(rows)
    if gate_up:   # tile rows: 32 gate, the same 32 up features, in turns
        order = np.arange(rows).reshape(2, -1, 32).transpose(1, 0, 2).reshape(-1)
    want = host(s)[:, order].reshape(E, rows // 128, 4, 32, K // 128, 4).transpose(0, 1, 4, 3, 2, 5)
    np.testing.assert_array_equal(host(packed).reshape(-1), want.reshape(-1))


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("T,H", [(1, 32), (3, 96), (1, 4096), (5, 1000 // 32 * 32), (2, 7168), (1, 32768), (700, 288),
                                 (650, 2048)])
@pytest.mark.parametrize("with_residual", [True, False])
def test_add_norm(moe, T, H, with_residual):
    torch = torch_()
    rng = np.random.default_rng(T * H)
    x, r = bf16(rng.standard_normal((T, H)) * 3), bf16(rng.standard_normal((T, H)))
    x[T // 2] = 0
    r[T // 2] = 0
    w = bf16(1 + 0.3 * rng.standard_normal(H))
    res = r if with_residual else None
    r_out, out = torch.empty_like(x), torch.empty_like(x)
    codes, scales = mx_buffers((T,), H)
    moe.moe_add_norm(x, res, w, 1e-6, r_out, out, codes, scales)
    v, n = mx_ref.norm(f64(x), f64(r) if with_residual else None, f64(w), 1e-6)
    want = (x.float() + r.float() if with_residual else x.float()).bfloat16()
    assert torch.equal(r_out, want)
    # bf16 rounds by at most 2^-8 of the value; the fp32 norm is off by (H/256 + 20) 2^-24 at most
    assert (np.abs(f64(out) - n) <= (2.0 ** -8 + (H / 256 + 20) * 2.0 ** -24) * np.abs(n)).all()
    c2, s2 = mx_buffers((T,), H)
    moe.moe_quantize_mx(out, c2, s2)
    assert torch.equal(codes, c2) and torch.equal(scales, s2)
    # the codes alone, the norm alone, and in place
    c3, s3 = mx_buffers((T,), H)
    moe.moe_add_norm(x, res, w, 1e-6, None, None, c3, s3)
    assert torch.equal(codes, c3) and torch.equal(scales, s3)
    x2, r2 = x.clone(), r.clone()
    moe.moe_add_norm(x2, r2 if with_residual else None, w, 1e-6, r2, x2)
    assert torch.equal(r2, r_out) and torch.equal(x2, out)


def test_add_norm_rows_do_not_depend_on_the_batch(moe):
    torch = torch_()
    rng = np.random.default_rng(5)
    x, r, w = bf16(rng.standard_normal((1500, 2080))), bf16(rng.standard_normal((1500, 2080))), bf16(np.ones(2080))
    a, b = torch.empty_like(x), torch.empty_like(x)
    moe.moe_add_norm(x, r, w, 1e-5, None, a)
    for t in (0, 7, 1499):
        moe.moe_add_norm(x[t:t + 1], r[t:t + 1], w, 1e-5, None, b[t:t + 1])
        assert torch.equal(a[t], b[t])


def test_add_norm_nan_and_inf_stay_in_their_row(moe):
    torch = torch_()
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    x[1, 3], x[2, 3] = float("nan"), float("inf")
    out = torch.empty_like(x)
    codes, scales = mx_buffers((4,), 64)
    moe.moe_add_norm(x, None, torch.ones(64, dtype=torch.bfloat16, device="cuda"), 0.0, None, out, codes, scales)
    assert torch.isnan(out[1]).all() and torch.isnan(out[2, 3]) and (out[2, 4:] == 0).all()
    assert (out[0] == 1).all() and (out[3] == 1).all()
    assert host(scales).tolist()[1:3] == [[255, 255], [255, 0]]


# ------------------------------------------------------------------ routing
ROUTES = [  # T, N, k, sigmoid, bias, groups, top_groups, top2, renorm
    (1, 1, 1, True, False, 1, 1, False, True),
    (3, 5, 5, False, True, 1, 1, False, False),
    (33, 8, 2, False, False, 1, 1, False, True),
    (64, 256, 8, True, True, 8, 4, True, True),
    (65, 128, 16, False, True, 4, 2, False, True),
    (40, 60, 6, True, False, 5, 3, True, False),
    (17, 250, 3, True, True, 25, 2, False, True),
    (9, 64, 4, False, False, 32, 7, True, True),
    (300, 96, 7, True, True, 3, 1, True, True),
    (301, 64, 5, False, True, 4, 2, True, True),
    (33, 256, 16, True, True, 2, 1, True, False),
    (70, 256, 16, False, True, 1, 1, False, True),
    (70, 128, 6, True, True, 32, 9, True, True),
    (70, 224, 12, True, False, 7, 2, False, False),     # a lane's list runs out (16 lanes, 12 slots)
    (90, 256, 16, True, True, 32, 2, True, True),       # every expert of two lanes
    (40, 16, 11, False, False, 2, 2, True, True),
]


def _route(moe, logits, bias, k, sigmoid, groups, top_groups, top2, renorm, scale=0.0):
    torch = torch_()
    T, N = logits.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    gate = torch.full((T, k), -7.0, device="cuda")
    sc = moe.make_scoring(moe.MOE_SCORE_SIGMOID if sigmoid else moe.MOE_SCORE_SOFTMAX, groups, top_groups,
                          moe.MOE_GROUP_TOP2_SUM if top2 else moe.MOE_GROUP_MAX, renorm, scale)
    moe.moe_route_scored(dict(hidden=128, num_experts=N, top_k=k, intermediate=128, block_size=8), sc,
                         torch.from_numpy(np.ascontiguousarray(logits, np.float32)).cuda(),
                         None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda(), idx, gate)
    return host(idx), host(gate).astype(np.float64)


@pytest.mark.parametrize("T,N,k,sigmoid,with_bias,groups,top_groups,top2,renorm", ROUTES)
def test_route_scored(moe, T, N, k, sigmoid, with_bias, groups, top_groups, top2, renorm):
    rng = np.random.default_rng(T * N + k)
    logits = rng.standard_normal((4 * T, N)).astype(np.float32)
    bias = (0.05 * rng.standard_normal(N)).astype(np.float32) if with_bias else None
    # rows whose choice hangs on less than fp32 resolves (scores are at most about 1) are left out
    keep = mx_ref.route(logits, bias, k, sigmoid, groups, top_groups, top2, renorm)[2] > 2e-6
    logits = logits[keep][:T]
    idx, gate, _ = mx_ref.route(logits, bias, k, sigmoid, groups, top_groups, top2, renorm, 2.5)
    got_idx, got_gate = _route(moe, logits, bias, k, sigmoid, groups, top_groups, top2, renorm, 2.5)
    np.testing.assert_array_equal(got_idx, idx)
    # exponential, division and a sum of up to 256 positive terms in fp32
    np.testing.assert_allclose(got_gate, gate, rtol=2e-6, atol=1e-12)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("top2", [True, False])
def test_route_ties_go_to_the_lower_index(moe, sigmoid, top2):
    # equal logits and a bias on a coarse grid: exact ties among experts and groups
    rng = np.random.default_rng(3)
    bias = rng.integers(0, 3, 64) * 0.25
    logits = np.zeros((1, 64))
    idx, gate, margin = mx_ref.route(logits, bias, 8, sigmoid, 8, 3, top2, True)
    assert margin[0] == 0
    got_idx, got_gate = _route(moe, logits, bias, 8, sigmoid, 8, 3, top2, True)
    np.testing.assert_array_equal(got_idx, idx)
    np.testing.assert_allclose(got_gate, gate, rtol=2e-6)


def test_route_masked_and_non_finite_logits(moe):
    inf, nan = np.inf, np.nan
    l = np.random.default_rng(0).standard_normal((8, 32)).astype(np.float32)
    l[0, :] = -inf                       # nothing is open
    l[1, 2:] = -inf                      # fewer open experts than slots
    l[2, ::2] = -inf
    l[3, 4] = nan
    l[4, :] = nan
    l[5, 9] = inf
    l[6, :] = np.finfo(np.float32).min   # masked with the type's lowest value
    l[7, 3:] = np.finfo(np.float32).min
    for sigmoid in (True, False):
        rows = [0, 1, 2, 6, 7] + ([3, 4, 5] if sigmoid else [])
        idx, gate, _ = mx_ref.route(l[rows], None, 4, sigmoid, renorm=True)
        got_idx, got_gate = _route(moe, l[rows], None, 4, sigmoid, 1, 1, False, True)
        np.testing.assert_array_equal(got_idx, idx)
        np.testing.assert_allclose(got_gate, gate, rtol=2e-6, atol=1e-12)
    # softmax of a row with a NaN or +inf: no answer but NaN; the indices stay in range and distinct
    got_idx, _ = _route(moe, l[[3, 4, 5]], None, 4, False, 4, 2, True, True)
    assert ((got_idx >= 0) & (got_idx < 32)).all() and (np.diff(got_idx, axis=1) > 0).all()


def test_route_takes_many_experts_of_one_lane(moe):
    """Ascending and descending runs: the best of a row sit next to each other, with and without ties."""
    base = np.linspace(-2, 2, 256)
    l = np.stack([base, base[::-1], np.repeat(np.linspace(2, -2, 32), 8), np.repeat(np.linspace(-2, 2, 64), 4)])
    for k in (5, 8, 13, 16):
        for sigmoid in (True, False):
            idx, gate, _ = mx_ref.route(l, None, k, sigmoid, renorm=True)
            got_idx, got_gate = _route(moe, l, None, k, sigmoid, 1, 1, False, True)
            np.testing.assert_array_equal(got_idx, idx)
            np.testing.assert_allclose(got_gate, gate, rtol=2e-6)


def test_route_rows_do_not_depend_on_the_batch(moe):
    l = np.random.default_rng(2).standard_normal((777, 160)).astype(np.float32)
    idx, gate = _route(moe, l, None, 6, False, 5, 2, True, True)
    for t in (0, 400, 776):
        i1, g1 = _route(moe, l[t:t + 1], None, 6, False, 5, 2, True, True)
        assert (i1 == idx[t]).all() and (g1 == gate[t]).all()


@pytest.mark.parametrize("N,groups", [(256, 8), (128, 4), (96, 3)])
def test_route_odd_rows_do_not_touch_their_neighbours(moe, N, groups):
    rng = np.random.default_rng(N)
    l = rng.standard_normal((41, N)).astype(np.float32)
    idx, gate = _route(moe, l, None, 5, True, groups, 2, True, True)
    odd = l.copy()
    odd[::3, 7] = np.nan
    odd[1::6, 9] = -np.inf
    bias = np.zeros(N)
    bias[3] = -np.inf            # an expert closed for every token
    i2, g2 = _route(moe, odd, None, 5, True, groups, 2, True, True)
    keep = np.isfinite(odd).all(1)
    assert (i2[keep] == idx[keep]).all() and (g2[keep] == gate[keep]).all()
    want, wg, _ = mx_ref.route(odd, None, 5, True, groups, 2, True, True)
    np.testing.assert_array_equal(i2, want)
    np.testing.assert_allclose(g2, wg, rtol=2e-6)
    i3, _ = _route(moe, l, bias, 5, True, groups, 2, True, True)
    np.testing.assert_array_equal(i3, mx_ref.route(l, bias, 5, True, groups, 2, True, True)[0])


# ------------------------------------------------------------------ expert FFN
class Layer:
    """MX weights of a layer: on the device, packed, and their values."""

    def __init__(self, moe, H, N, k, I, B, Is=0, seed=0, **cfg):
        torch = torch_()
        rng = np.random.default_rng(seed)
        self.cfg = moe.make_config(H, N, k, I, B, shared_intermediate=Is, **cfg)
        self.H, self.N, self.k, self.I, self.B, self.Is = H, N, k, I, B, Is
        self.moe = moe
        self.dev, self.val = [], []
        for n, rows, K, gate_up in ((N, 2 * I, H, True), (N, H, I, False), (1, 2 * Is, H, True), (1, H, Is, False)):
            if rows == 0 or K == 0:
                self.dev += [None, None]
                self.val.append(None)
                continue
            c, s = mx_ref.quantize(rng.standard_normal((n, rows, K)) * 0.05)
            self.val.append(mx_ref.dequantize(c, s))
            sd = torch.from_numpy(s).cuda()
            packed = torch.empty_like(sd)
            moe.moe_pack_scales_mx(sd, packed, gate_up)
            self.dev += [torch.from_numpy(c).cuda(), packed]

    def dispatch(self, idx):
        """Layout of routes idx [T, k] (torch int32)."""
        torch, moe = torch_(), self.moe
        T = idx.shape[0]
        R, rows = T * self.k, moe.moe_max_padded_rows(self.cfg, T)
        e = dict(device="cuda", dtype=torch.int32)
        d = dict(kept=torch.empty(R, dtype=torch.uint8, device="cuda"), pos=torch.empty(R, **e),
                 ids=torch.full((rows,), -9, **e), blocks=torch.full((moe.moe_max_blocks(self.cfg, T),), -9, **e),
                 npad=torch.zeros(1, **e), counts=torch.empty(self.N, **e), dropped=torch.zeros(1, **e))
        ws = moe.workspace(self.cfg, T)
        moe.moe_dispatch_align(self.cfg, idx, d["kept"], d["pos"], d["ids"], d["blocks"], d["npad"], d["counts"],
                               d["dropped"], ws)
        return d

    def ffn(self, codes, scales, d, ws=None):
        torch, moe = torch_(), self.moe
        T = codes.shape[0]
        y = torch.full((moe.moe_max_padded_rows(self.cfg, T), self.H), 7.0, dtype=torch.bfloat16, device="cuda")
        ysh = torch.full((T, self.H), 7.0, dtype=torch.bfloat16, device="cuda") if self.Is else None
        ws = moe.workspace_mx(self.cfg, T) if ws is None else ws
        moe.moe_clear_device_status(ws)
        moe.moe_expert_ffn_mx(self.cfg, codes, scales, *self.dev, d["ids"], d["blocks"], d["npad"], y, ysh, ws)
        torch.cuda.synchronize()
        assert moe.moe_get_device_status(ws) == 0
        return y, ysh


def _tokens(rng, T, H):
    x = rng.standard_normal((T, H)) * (1 + 9 * (rng.random(H) < 0.02))
    return mx_ref.quantize(x)


def _check_rows(L, y, xv, d, rows=None):
    ids, blocks, P = host(d["ids"]), host(d["blocks"]), int(host(d["npad"])[0])
    R = xv.shape[0] * L.k
    got = f64(y)
    for e in range(L.N):
        at = np.flatnonzero((np.repeat(blocks[:P // L.B], L.B) == e) & (ids[:P] < R))
        if rows is not None:
            at = at[np.isin(at, rows)]
        if at.size:
            ref, tol = mx_ref.ffn_rows(xv[ids[at] // L.k], L.val[0][e], L.val[1][e])
            bad = np.abs(got[at] - ref) > tol
            assert not bad.any(), (e, int(bad.sum()), float(np.abs(got[at] - ref).max()))
    pad = np.setdiff1d(np.arange(len(got)), np.flatnonzero(ids[:P] < R))
    assert (got[pad] == 7.0).all(), "padding rows are not written"


FFNS = [  # T, H, N, k, I, B, Is
    (1, 128, 1, 1, 128, 8, 0),
    (1, 256, 8, 2, 384, 64, 128),
    (5, 384, 4, 3, 256, 16, 256),
    (33, 512, 16, 2, 384, 8, 128),       # tiles of 32 rows, several an expert
    (100, 256, 4, 2, 128, 16, 0),
    (33, 640, 3, 1, 128, 128, 0),
    (130, 128, 8, 2, 256, 8, 128),
    (257, 256, 2, 2, 256, 32, 384),
    (400, 384, 5, 2, 640, 8, 0),
    (1500, 768, 64, 4, 512, 8, 0),       # enough tiles for the wide work items
    (2300, 640, 24, 4, 640, 16, 0),      # the same, an odd number of 128-row weight tiles
]


@pytest.mark.parametrize("T,H,N,k,I,B,Is", FFNS)
def test_expert_ffn(moe, T, H, N, k, I, B, Is):
    torch = torch_()
    rng = np.random.default_rng(T + H + N)
    L = Layer(moe, H, N, k, I, B, Is, seed=T)
    c, s = _tokens(rng, T, H)
    idx = np.sort(np.argsort(rng.random((T, N)) + rng.random(N), axis=1)[:, :k], axis=1).astype(np.int32)
    d = L.dispatch(torch.from_numpy(idx).cuda())
    y, ysh = L.ffn(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), d)
    xv = mx_ref.dequantize(c, s)
    _check_rows(L, y, xv, d)
    if Is:
        ref, tol = mx_ref.ffn_rows(xv, L.val[2][0], L.val[3][0])
        assert (np.abs(f64(ysh) - ref) <= tol).all()


def test_expert_ffn_long_reductions(moe):
    """K past 32 scale chunks in both products; one expert takes every token."""
    torch = torch_()
    rng = np.random.default_rng(8)
    L = Layer(moe, 4224, 3, 1, 4480, 8, seed=3)
    c, s = _tokens(rng, 140, 4224)
    d = L.dispatch(torch.full((140, 1), 1, dtype=torch.int32, device="cuda"))
    y, _ = L.ffn(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), d)
    _check_rows(L, y, mx_ref.dequantize(c, s), d)


def test_expert_ffn_nan_and_zero_rows(moe):
    torch = torch_()
    L = Layer(moe, 256, 2, 1, 128, 8, seed=4)
    x = np.random.default_rng(4).standard_normal((6, 256))
    x[1], x[3, 7], x[4] = 0, np.nan, x[4] * 2.0 ** 100    # zero row, NaN row, overflowing row
    c, s = mx_ref.quantize(x)
    d = L.dispatch(torch.tensor([[0], [0], [0], [0], [0], [1]], dtype=torch.int32, device="cuda"))
    y, _ = L.ffn(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), d)
    got = f64(y)[:5]
    assert np.isnan(got[3]).all() and (got[1] == 0).all() and np.isfinite(got[[0, 2]]).all()
    ref, tol = mx_ref.ffn_rows(mx_ref.dequantize(c, s)[[0, 2]], L.val[0][0], L.val[1][0])
    assert (np.abs(got[[0, 2]] - ref) <= tol).all()


@pytest.mark.parametrize("N", [32, 16, 256])
def test_expert_ffn_rows_do_not_depend_on_the_batch(moe, N):
    """A token alone (operands swapped) and in a batch of many tiles (wide items; with 16
    experts CTA pairs; with 256 tiles of 25 rows): the same bits."""
    torch = torch_()
    rng = np.random.default_rng(11)
    L = Layer(moe, 768, N, 4, 640, 16, Is=256, seed=6)
    T = 1600
    c, s = (torch.from_numpy(v).cuda() for v in _tokens(rng, T, 768))
    idx = torch.from_numpy(np.sort(np.argsort(rng.random((T, N)), axis=1)[:, :4], axis=1).astype(np.int32)).cuda()
    d = L.dispatch(idx)
    y, ysh = L.ffn(c, s, d)
    few = slice(100, 170)   # 64-column items
    df = L.dispatch(idx[few].contiguous())
    yf, yshf = L.ffn(c[few].clone(), s[few].clone(), df)
    for j in range(0, 280, 7):
        assert torch.equal(y[d["pos"][400 + j]], yf[df["pos"][j]])
    assert torch.equal(ysh[few], yshf)
    for t in (0, 3, 801, 1599):
        d1 = L.dispatch(idx[t:t + 1].contiguous())
        y1, ysh1 = L.ffn(c[t:t + 1].clone(), s[t:t + 1].clone(), d1)   # a copy: pointers are 16-byte aligned
        for j in range(4):
            assert torch.equal(y[d["pos"][4 * t + j]], y1[d1["pos"][j]])
        assert torch.equal(ysh[t], ysh1[0])
    again, _ = L.ffn(c, s, d)
    assert torch.equal(again, y)


@pytest.mark.parametrize("T", [8300, 8301])
def test_expert_ffn_long_block_list(moe, T):
    """More blocks than one round of the front's loads takes; counts that four does not divide."""
    torch = torch_()
    rng = np.random.default_rng(T)
    L = Layer(moe, 128, 16, 4, 128, 8, seed=15)
    c, s = _tokens(rng, T, 128)
    idx = np.sort(np.argsort(rng.random((T, 16)), axis=1)[:, :4], axis=1).astype(np.int32)
    d = L.dispatch(torch.from_numpy(idx).cuda())
    y, _ = L.ffn(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), d)
    assert int(d["npad"][0]) > 4096 * L.B
    _check_rows(L, y, mx_ref.dequantize(c, s), d)


def test_expert_ffn_list_with_holes(moe):
    """A caller's list may hold ids out of range between routes and end in blocks without a
    route: the routed rows are what they are without them."""
    torch = torch_()
    L = Layer(moe, 256, 4, 2, 128, 64, seed=13)
    T = 60
    rng = np.random.default_rng(13)
    c, s = (torch.from_numpy(v).cuda() for v in _tokens(rng, T, 256))
    idx = torch.from_numpy(np.sort(np.argsort(rng.random((T, 4)), axis=1)[:, :2], axis=1).astype(np.int32)).cuda()
    d = L.dispatch(idx)
    y, _ = L.ffn(c, s, d)
    ids, P = d["ids"].clone(), int(d["npad"][0])
    keep = (ids >= 0) & (ids < 2 * T)
    ids[1:P:9] = 2 * T                    # holes
    ids[3:P:11] = -5
    d2 = dict(d, ids=ids)
    y2, _ = L.ffn(c, s, d2)
    same = keep & (ids == d["ids"]) & (torch.arange(len(ids), device="cuda") < P)
    assert torch.equal(y2[same], y[same])


def test_expert_ffn_bad_block_list_does_no_work(moe):
    torch = torch_()
    L = Layer(moe, 128, 4, 1, 128, 8, seed=9)
    c, s = (torch.from_numpy(v).cuda() for v in _tokens(np.random.default_rng(1), 40, 128))
    d = L.dispatch(torch.arange(40, device="cuda", dtype=torch.int32).reshape(40, 1) % 4)
    d["blocks"][1] = 3                                   # unsorted
    y = torch.full((moe.moe_max_padded_rows(L.cfg, 40), 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = moe.workspace_mx(L.cfg, 40)
    moe.moe_clear_device_status(ws)
    moe.moe_expert_ffn_mx(L.cfg, c, s, *L.dev, d["ids"], d["blocks"], d["npad"], y, None, ws)
    torch.cuda.synchronize()
    assert moe.moe_get_device_status(ws) & moe.MOE_DEV_ERR_BAD_BLOCKS
    assert (y == 7.0).all()


@pytest.mark.parametrize("T,N,k,Is", [
    (9, 8, 2, 1024),      # swapped operands, also the shared expert
    (70, 2, 1, 0),        # 64-column items
    (300, 8, 2, 0),       # wider ones
    (600, 8, 2, 14336)])  # CTA pairs
def test_expert_ffn_waits_run_out_and_report(moe, T, N, k, Is):
    """With a 1 ns limit a wait that one suspension does not see through gives up (the longest
    are those for a tile of a 14336-deep reduction): the status says so, nothing hangs, and the
    next call with the default limits gives the usual bits."""
    torch = torch_()
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    H, I, B = 4096, 14336, 16

    def rand(*shape, low=0, high=256):
        return torch.randint(low, high, shape, generator=g, device="cuda", dtype=torch.uint8)
    L = Layer.__new__(Layer)
    L.cfg, L.moe = moe.make_config(H, N, k, I, B, shared_intermediate=Is), moe
    L.H, L.N, L.k, L.I, L.B, L.Is = H, N, k, I, B, Is
    L.dev = [rand(N, 2 * I, H // 2), rand(N, 2 * I, H // 32, low=118, high=122),
             rand(N, H, I // 2), rand(N, H, I // 32, low=118, high=122)]
    L.dev += [rand(1, 2 * Is, H // 2), rand(1, 2 * Is, H // 32, low=118, high=122),
              rand(1, H, Is // 2), rand(1, H, Is // 32, low=118, high=122)] if Is else [None] * 4
    c, s = rand(T, H // 2), rand(T, H // 32, low=124, high=128)
    idx = torch.rand(T, N, generator=g, device="cuda").topk(k, 1).indices.sort(1).values.int()
    d = L.dispatch(idx)
    y, ysh = L.ffn(c, s, d)
    ws, y2 = moe.workspace_mx(L.cfg, T), torch.empty_like(y)
    L.cfg.debug_wait_ns = 1
    for _ in range(2):
        moe.moe_clear_device_status(ws)
        moe.moe_expert_ffn_mx(L.cfg, c, s, *L.dev, d["ids"], d["blocks"], d["npad"], y2,
                              None if ysh is None else torch.empty_like(ysh), ws)
        torch.cuda.synchronize()
        assert moe.moe_get_device_status(ws) & moe.MOE_DEV_ERR_TIMEOUT
    L.cfg.debug_wait_ns = 0
    y3, ysh3 = L.ffn(c, s, d, ws)
    assert torch.equal(y3.view(torch.int16), y.view(torch.int16))
    assert ysh is None or torch.equal(ysh3.view(torch.int16), ysh.view(torch.int16))


def test_expert_ffn_on_another_stream(moe):
    torch = torch_()
    L = Layer(moe, 256, 4, 2, 256, 8, seed=10)
    c, s = (torch.from_numpy(v).cuda() for v in _tokens(np.random.default_rng(2), 70, 256))
    idx = torch.tensor([[0, 3], [1, 2]], dtype=torch.int32, device="cuda").repeat(35, 1)
    d = L.dispatch(idx)
    y, _ = L.ffn(c, s, d)
    st = torch.cuda.Stream()
    ws = moe.workspace_mx(L.cfg, 70)
    y2 = torch.full_like(y, 7.0)
    st.wait_stream(torch.cuda.current_stream())
    moe.moe_expert_ffn_mx(L.cfg, c, s, *L.dev, d["ids"], d["blocks"], d["npad"], y2, None, ws, stream=st)
    st.synchronize()
    assert torch.equal(y, y2)


# ------------------------------------------------------------------ the layer
@pytest.mark.parametrize("T,with_residual,cf,Is", [(1, True, 0.0, 0), (77, False, 0.0, 128), (500, True, 1.0, 0)])
def test_forward_is_its_stages(moe, T, with_residual, cf, Is):
    torch = torch_()
    H, N, k, I, B = 256, 16, 4, 128, 8
    L = Layer(moe, H, N, k, I, B, Is, seed=12, capacity_factor=cf)
    rng = np.random.default_rng(T)
    x, r = bf16(rng.standard_normal((T, H))), bf16(rng.standard_normal((T, H))) if with_residual else None
    nw, wg = bf16(1 + 0.1 * rng.standard_normal(H)), bf16(rng.standard_normal((H, N)) / 16)
    sb = torch.from_numpy((0.1 * rng.standard_normal(N)).astype(np.float32)).cuda()
    sc = moe.make_scoring(moe.MOE_SCORE_SIGMOID, 4, 2, moe.MOE_GROUP_TOP2_SUM, True, 2.5)
    out, ws = torch.empty_like(x), moe.workspace_mx(L.cfg, T)
    moe.moe_clear_device_status(ws)
    moe.moe_forward_mx(L.cfg, sc, x, r, nw, 1e-6, wg, None, sb, *L.dev, out, ws)
    torch.cuda.synchronize()
    assert moe.moe_get_device_status(ws) == 0

    ws0 = moe.workspace(L.cfg, T)
    v, n = torch.empty_like(x), torch.empty_like(x)
    codes, scales = mx_buffers((T,), H)
    moe.moe_add_norm(x, r, nw, 1e-6, v, n, codes, scales)
    logits = torch.empty(T, N, device="cuda")
    moe.moe_router_logits(L.cfg, n, wg, None, logits, ws0)
    idx, gate = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_route_scored(L.cfg, sc, logits, sb, idx, gate)
    d = L.dispatch(idx)
    y, ysh = L.ffn(codes, scales, d)
    want = torch.empty_like(x)
    moe.moe_combine(L.cfg, v, gate, d["kept"], d["pos"], y, ysh, want)
    assert torch.equal(out, want)
    if cf:
        assert int(d["dropped"][0]) > 0
