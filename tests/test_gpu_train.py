"""The training step's operators against their formulas in 64 bits, at the sizes and layouts where they can go wrong."""
import pytest

from tests.test_gpu_mx import moe, torch_  # noqa: F401

pytestmark = pytest.mark.gpu


def _gen(seed):
    g = torch_().Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0):
    return torch_().randn(*shape, generator=g, device="cuda").mul_(scale).bfloat16()


def _gemm(moe, G, x, w, gather, transposed, cfg=None, ws=None, fill=7.0):
    torch = torch_()
    F = w.shape[1] if transposed else w.shape[2]
    cfg = cfg or moe.make_config(128, G.N, G.k, 128, G.B)
    ws = moe.workspace_grouped(cfg, G.T) if ws is None else ws
    y = torch.full((G.rows, F), fill, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm(cfg, G.T, x, w, G.ids if gather else None, G.dcounts, y, ws, gather=gather, transposed=transposed)
    assert moe.moe_get_device_status(ws) == 0
    return y


LAYOUTS = [  # T, N, k, B, skew, idle experts
    (1, 1, 1, 8, 0, ()), (1, 8, 2, 128, 0, ()), (64, 8, 2, 8, 0, (3,)), (33, 5, 3, 16, 0, (0,)),
    (300, 3, 1, 64, 0.9, (2,)), (257, 16, 4, 32, 0.5, (15, 7)), (1000, 6, 2, 8, 0.97, ()), (130, 256, 6, 8, 0, (255,))]
SIZES = [(8, 8), (128, 512), (72, 200), (328, 1000), (1000, 264), (264, 8), (8, 1032)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("layout", range(len(LAYOUTS)))
def test_grouped_gemm(moe, layout, transposed, gather):
    from tests import train_ref as R
    T, N, k, B, skew, idle = LAYOUTS[layout]
    G = R.Groups(T, N, k, B, seed=layout, skew=skew, idle=idle)
    for K, F in SIZES:
        g = _gen(K + F)
        x = _randn(g, T, K) if gather else G.grouped(K, g)
        w = _randn(g, *((N, F, K) if transposed else (N, K, F)), scale=0.1)
        y = _gemm(moe, G, x, w, gather, transposed)
        want, mag = R.gemm(G, x, w, gather, transposed)
        assert (y[~G.real] == 7).all()
        R.check(y[G.real], want[G.real], R.BF * want[G.real].abs() + R.sum_tol(K) * mag[G.real], (K, F))


def test_a_row_does_not_depend_on_the_batch(moe):
    torch = torch_()
    from tests import train_ref as R
    K, F, N = 1096, 520, 4
    g = _gen(3)
    w, wt, row = _randn(g, N, K, F, scale=0.1), _randn(g, N, F, K, scale=0.1), _randn(g, 1, K)
    seen = {False: [], True: []}
    for T, B, skew in ((1, 8, 0), (20, 8, 0.9), (100, 128, 0.5), (900, 16, 0.9)):
        G = R.Groups(T, N, 1, B, seed=T, skew=skew)
        x = _randn(g, T, K)
        x[T // 2] = row
        p = int((G.ids == T // 2).nonzero()[0])
        e = next(e for e in range(N) if G.start[e] <= p < G.start[e] + G.counts[e])
        for transposed in (False, True):
            weights = (wt if transposed else w)[e:e + 1].expand(N, -1, -1).contiguous()
            weights = torch.where(torch.arange(N, device="cuda").reshape(-1, 1, 1) == e, (wt if transposed else w)[:1],
                                  weights)
            seen[transposed].append(_gemm(moe, G, x, weights, True, transposed)[p])
            xp = torch.full((G.rows, K), float("nan"), dtype=torch.bfloat16, device="cuda")
            xp[G.real] = x[G.ids[G.real].long()]
            seen[transposed].append(_gemm(moe, G, xp, weights, False, transposed)[p])
    for rows in seen.values():
        assert all(torch.equal(rows[0], r) for r in rows[1:])


@pytest.mark.parametrize("form", ["fp32", "add", "in place", "bf16"])
@pytest.mark.parametrize("layout", range(len(LAYOUTS)))
def test_grouped_wgrad(moe, layout, form):
    torch = torch_()
    from tests import train_ref as R
    T, N, k, B, skew, idle = LAYOUTS[layout]
    G = R.Groups(T, N, k, B, seed=layout, skew=skew, idle=idle)
    cfg = moe.make_config(128, N, k, 128, B)
    ws = moe.workspace_grouped(cfg, T)
    n = torch.tensor(G.counts, device="cuda").reshape(-1, 1, 1).double()
    for i, (K, F) in enumerate(SIZES):
        if N * K * F > 2 ** 26:
            continue
        g = _gen(K + F)
        gx, gd = [(False, False), (True, False), (False, True), (True, True)][(i + layout) % 4]
        x = _randn(g, T, K) if gx else G.grouped(K, g)
        dy = _randn(g, T, F) if gd else G.grouped(F, g)
        dw = torch.full((N, K, F), 7.0, dtype=torch.bfloat16 if form == "bf16" else torch.float32, device="cuda")
        add = None
        if form in ("add", "in place"):
            add = torch.randn(N, K, F, generator=g, device="cuda")
        want, mag = R.wgrad(G, x, dy, gx, gd)
        if add is not None:
            want = want + add.double()
        if form == "in place":
            dw = add
        moe.moe_grouped_wgrad(cfg, T, x, dy, G.ids, G.dcounts, dw, ws, dw_add=add, gather_x=gx, gather_dy=gd)
        assert moe.moe_get_device_status(ws) == 0
        step = R.BF if form == "bf16" else 2.0 ** -23   # the sum's rounding, and the sum with dw_add
        R.check(dw, want, step * want.abs() + R.sum_tol(n) * mag, (K, F))
        again = torch.empty_like(dw)
        if form in ("fp32", "bf16"):
            moe.moe_grouped_wgrad(cfg, T, x, dy, G.ids, G.dcounts, again, ws, gather_x=gx, gather_dy=gd)
            assert torch.equal(again, dw)


def test_ids_outside_read_zeros(moe):
    torch = torch_()
    from tests import train_ref as R
    T, N, k, B, K, F = 90, 3, 2, 8, 136, 264
    G = R.Groups(T, N, k, B)
    g = _gen(1)
    x, w, dy = _randn(g, T, K), _randn(g, N, K, F, scale=0.1), G.grouped(F, g)
    gone = G.real & (torch.rand(G.rows, generator=g, device="cuda") < 0.3)
    y0 = _gemm(moe, G, x, w, True, False)
    ids = G.ids.clone()
    ids[gone] = torch.tensor([-1, G.R, 2 ** 31 - 1, -2 ** 31, G.R + 7], dtype=torch.int32,
                             device="cuda").repeat(G.rows)[:G.rows][gone]
    G.ids = ids
    y = _gemm(moe, G, x, w, True, False)
    assert (y[gone] == 0).all() and torch.equal(y[G.real & ~gone], y0[G.real & ~gone]) and (y[~G.real] == 7).all()
    cfg = moe.make_config(128, N, k, 128, B)
    ws = moe.workspace_grouped(cfg, T)
    dw = torch.empty(N, K, F, device="cuda")
    moe.moe_grouped_wgrad(cfg, T, x, dy, ids, G.dcounts, dw, ws, gather_x=True)
    G2 = R.Groups(T, N, k, B)
    dy2 = dy.clone()
    dy2[gone] = 0
    want, mag = R.wgrad(G2, x, dy2, True, False)
    R.check(dw, want, 2.0 ** -23 * want.abs() + R.sum_tol(max(G.counts)) * mag)


@pytest.mark.parametrize("counts", [[-1, 4, 4], [200, 3, 3], [2 ** 31 - 1, 2 ** 31 - 1, 2], [100, 100, 100]])
def test_bad_counts_are_reported(moe, counts):
    torch = torch_()
    from tests import train_ref as R
    T, N, k, B, K, F = 90, 3, 2, 8, 136, 264
    G = R.Groups(T, N, k, B)
    g = _gen(1)
    x, w, dy = _randn(g, T, K), _randn(g, N, K, F), G.grouped(F, g)
    bad = torch.tensor(counts, dtype=torch.int32, device="cuda")
    cfg = moe.make_config(128, N, k, 128, B)
    ws = moe.workspace_grouped(cfg, T)
    y = torch.full((G.rows, F), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((N, K, F), 7.0, device="cuda")
    moe.moe_grouped_gemm(cfg, T, x, w, G.ids, bad, y, ws, gather=True)
    assert moe.moe_get_device_status(ws) == moe.MOE_DEV_ERR_BAD_BLOCKS and (y == 7).all()
    moe.moe_clear_device_status(ws)
    moe.moe_grouped_wgrad(cfg, T, x, dy, G.ids, bad, dw, ws, gather_x=True)
    assert moe.moe_get_device_status(ws) == moe.MOE_DEV_ERR_BAD_BLOCKS and (dw == 7).all()


def test_offsets_past_32_bits(moe):
    """Grouped tensors of more than 2^31 elements, the rows at their ends."""
    torch = torch_()
    from tests import train_ref as R
    T, K, F = 140_001, 8, 16384
    G = R.Groups(T, 1, 1, 8)
    g = _gen(2)
    x, w = _randn(g, T, K), _randn(g, 1, K, F)
    y = _gemm(moe, G, x, w, True, False)
    assert y.numel() > 2 ** 31
    for at in (slice(0, 50), slice(131_000, 131_100), slice(T - 50, T)):
        want = x[at].double() @ w[0].double()
        R.check(y[at], want, R.BF * want.abs() + R.sum_tol(K) * (x[at].double().abs() @ w[0].double().abs()))
    cfg = moe.make_config(128, 1, 1, 128, 8)
    ws = moe.workspace_grouped(cfg, T)
    dw = torch.empty(1, K, F, device="cuda")
    moe.moe_grouped_wgrad(cfg, T, x, y, G.ids, G.dcounts, dw, ws, gather_x=True)
    for at in (slice(0, 64), slice(F - 64, F)):
        want = x.double().t() @ y[:T, at].double()
        R.check(dw[0, :, at], want, 2.0 ** -23 * want.abs() + R.sum_tol(T) * (x.double().abs().t() @ y[:T, at].double().abs()))


def _swiglu_case(moe, G, I, seed, gates=True, scale=2.0):
    torch = torch_()
    g = _gen(seed)
    cfg = moe.make_config(128, G.N, G.k, I, G.B)
    gate = torch.rand(G.T, G.k, generator=g, device="cuda") + 0.05 if gates else None
    return cfg, G.grouped(2 * I, g, scale=scale), G.grouped(I, g), gate


# relative error of 1 / (1 + e^-g) up to |g| = 20: the fast exponential is off by (2 + 1.173 |g|) 2^-23, the
# division by 2^-22; a few products and sums more
SWIGLU = 2.0 ** -17


@pytest.mark.parametrize("gates", [True, False])
@pytest.mark.parametrize("layout", range(len(LAYOUTS)))
def test_swiglu(moe, layout, gates):
    torch = torch_()
    from tests import train_ref as R
    T, N, k, B, skew, idle = LAYOUTS[layout]
    G = R.Groups(T, N, k, B, seed=layout, skew=skew, idle=idle)
    for I in (128, 384, 2176):
        cfg, gu, da, gate = _swiglu_case(moe, G, I, I, gates)
        a, a2, dgu = (torch.full((G.rows, n), 7.0, dtype=torch.bfloat16, device="cuda") for n in (I, I, 2 * I))
        dgate = torch.full((T, k), 7.0, device="cuda")
        moe.moe_swiglu(cfg, T, gu, gate, G.ids, G.num_padded, a)
        moe.moe_swiglu_backward(cfg, T, gu, gate, da, G.ids, G.num_padded, dgu, dgate, a2)
        assert torch.equal(a, a2) and (a[~G.real] == 7).all() and (dgu[~G.real] == 7).all()
        r = G.ids[G.real].long()
        gg, u = gu[G.real].double().split(I, -1)
        d = da[G.real].double()
        w = gate.flatten()[r].double().unsqueeze(-1) if gates else torch.ones(r.numel(), 1, dtype=R.F64, device="cuda")
        want = R.swiglu(gg, u, w)
        R.check(a[G.real], want, (R.BF + SWIGLU) * want.abs() + 2.0 ** -130)
        dg, du, dw = R.swiglu_backward(gg, u, w, d)
        s = torch.sigmoid(gg)
        R.check(dgu[G.real][:, :I], dg, R.BF * dg.abs() + SWIGLU * (w * d * u).abs() * s * (1 + gg.abs()) + 2.0 ** -130)
        R.check(dgu[G.real][:, I:], du, (R.BF + SWIGLU) * du.abs() + 2.0 ** -130)
        R.check(dgate.flatten()[r], dw, 2 * SWIGLU * (d * gg * s * u).abs().sum(-1) + 2.0 ** -130)
        if G.R == r.numel():
            # in place, and without the optional outputs
            da2, gu2 = da.clone(), gu.clone()
            moe.moe_swiglu_backward(cfg, T, gu2, gate, da2, G.ids, G.num_padded, gu2, None, da2)
            assert torch.equal(gu2[G.real], dgu[G.real]) and torch.equal(da2[G.real], a[G.real])


def test_swiglu_at_the_ends(moe):
    """Gates far from zero, infinities and NaN: the fp32 formula's values."""
    torch = torch_()
    from tests import train_ref as R
    G = R.Groups(8, 1, 1, 8)
    I = 128
    cfg, gu, da, gate = _swiglu_case(moe, G, I, 0)
    ends = [0.0, -0.0, 88.0, -88.0, 1e4, -1e4, 3e38, -3e38]
    for i, v in enumerate(ends):
        gu[:, i] = v
    gu[:, I + 20], gu[:, 21], gu[:, I + 22] = float("inf"), float("nan"), 0.0
    a, dgu = torch.empty_like(da), torch.empty_like(gu)
    moe.moe_swiglu_backward(cfg, 8, gu, gate, da, G.ids, G.num_padded, dgu, None, a)
    r = G.ids[:8].long()
    w, (g, u), d = gate.flatten()[r].unsqueeze(-1), gu[:8].float().split(I, -1), da[:8].float()
    s = 1 / (1 + torch.exp(-g))
    want = g * s * (w * u)
    assert torch.equal(torch.isnan(a[:8]), torch.isnan(want)) and torch.equal(torch.isinf(a[:8]), torch.isinf(want.bfloat16()))
    dg, du = d * (w * u) * (s * (1 + g * (1 - s))), w * d * (g * s)
    for got, ref in ((dgu[:8, :I], dg), (dgu[:8, I:], du)):
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert (dgu[:8, [5, 7]] == 0).all() and (a[:8, [0, 1, 5, 7]] == 0).all()   # silu and its slope far below zero
    assert torch.isfinite(dgu[:8, :8]).all()


NORMS = [(1, 8), (1, 4096), (3, 40), (37, 2048), (100, 264), (5, 32768), (700, 1096), (650, 8712), (2049, 4096), (129, 7168),
         (3, 16392)]


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("offset", [0.0, 30.0])
def test_add_layer_norm(moe, T, H, offset):
    torch = torch_()
    from tests import train_ref as R
    g = _gen(T + H)
    x, r = (_randn(g, T, H).float() + offset).bfloat16(), _randn(g, T, H)
    w, b = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).bfloat16(), _randn(g, H)
    for res, bias in ((r, b), (None, b), (r, None)):
        out, r_out = torch.empty_like(x), torch.empty_like(x)
        moe.moe_add_layer_norm(x, res, w, bias, 1e-5, r_out, out)
        v = x.double() + (r.double() if res is not None else 0)
        bd = b.double() if bias is not None else torch.zeros(H, dtype=R.F64, device="cuda")
        R.check(r_out, v, (R.BF + 2.0 ** -23) * v.abs())
        d = v - v.mean(-1, keepdim=True)
        n = d / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-5)
        inv = n.abs().amax(-1, keepdim=True) / d.abs().amax(-1, keepdim=True).clamp(min=1e-30)
        want = n * w.double() + bd
        # fp32 sums of a fixed tree (8 + 5 + 7 + 5 additions), a few roundings more: 64 of 2^-24, and the mean's
        # error carried into every deviation
        slack = 2.0 ** -18 * ((n * w.double()).abs() + bd.abs() + inv * v.abs().mean(-1, keepdim=True) * w.double().abs())
        R.check(out, want, R.BF * want.abs() + slack)
        # in place: the same bits
        x2 = x.clone()
        r2 = r.clone() if res is not None else torch.empty_like(x)
        moe.moe_add_layer_norm(x2, r2 if res is not None else None, w, bias, 1e-5, r2, x2)
        assert torch.equal(x2, out) and torch.equal(r2, r_out)


def test_a_norm_does_not_depend_on_the_batch(moe):
    torch = torch_()
    g = _gen(9)
    for H in (2048, 4104):
        x, w, b = _randn(g, 2000, H), _randn(g, H), _randn(g, H)
        out, one = torch.empty_like(x), torch.empty(1, H, dtype=torch.bfloat16, device="cuda")
        moe.moe_add_layer_norm(x, None, w, b, 1e-5, None, out)
        moe.moe_add_layer_norm(x[1234:1235].clone(), None, w, b, 1e-5, None, one)
        assert torch.equal(out[1234:1235], one)
        dout, dx = _randn(g, 2000, H), torch.empty_like(x)
        ws = moe.workspace_norm_backward(2000, H)
        for centre in (True, False):
            moe.moe_norm_backward(x, dout, None, w, 1e-5, dx, None, None, ws, centre=centre)
            moe.moe_norm_backward(x[1234:1235].clone(), dout[1234:1235].clone(), None, w, 1e-5, one, None, None, ws,
                                  centre=centre)
            assert torch.equal(dx[1234:1235], one)


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("centre", [True, False])
@pytest.mark.parametrize("offset", [0.0, 30.0])
def test_norm_backward(moe, T, H, centre, offset):
    torch = torch_()
    from tests import train_ref as R
    g = _gen(T + H)
    v, dout, dres = (_randn(g, T, H).float() + offset).bfloat16(), _randn(g, T, H), _randn(g, T, H)
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).bfloat16()
    ws = moe.workspace_norm_backward(T, H)
    for res in (dres, None):
        dx, dw, db = torch.empty_like(v), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
        moe.moe_norm_backward(v, dout, res, w, 1e-5, dx, dw, db, ws, centre=centre)
        r = res.double() if res is not None else torch.zeros(T, H, dtype=R.F64, device="cuda")
        want, want_w, want_b, mag, mag_w, mag_b = R.norm_backward(v.double(), dout.double(), r, w.double(), 1e-5, centre)
        R.check(dx, want, R.BF * want.abs() + 2.0 ** -17 * mag, "dx")
        # a column's rows are summed in slabs, then the slabs: at most T / 128 + 160 additions in turn
        adds = (T / 128 + 160 + 64) * 2.0 ** -24
        R.check(dw, want_w, adds * mag_w, "dweight")
        R.check(db, want_b, adds * mag_b, "dbias")
        dx2, dw2, db2 = (res.clone() if res is not None else torch.empty_like(v)), torch.empty_like(dw), torch.empty_like(db)
        moe.moe_norm_backward(v, dout, dx2 if res is not None else None, w, 1e-5, dx2, dw2, None, ws, centre=centre)
        moe.moe_norm_backward(v, dout, res, w, 1e-5, torch.empty_like(v), None, db2, ws, centre=centre)
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


def test_norm_backward_offsets_past_32_bits(moe):
    torch = torch_()
    from tests import train_ref as R
    T, H = 150_001, 14336
    g = _gen(4)
    v, dout = _randn(g, T, H), _randn(g, T, H)
    assert v.numel() > 2 ** 31
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    dx, dw, db = torch.empty_like(v), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    moe.moe_norm_backward(v, dout, None, w, 1e-5, dx, dw, db, moe.workspace_norm_backward(T, H))
    for at in (slice(0, 3), slice(149_790, 149_800), slice(T - 3, T)):
        want, _, _, mag, _, _ = R.norm_backward(v[at].double(), dout[at].double(), torch.zeros_like(v[at]).double(),
                                                w.double(), 1e-5, True)
        R.check(dx[at], want, R.BF * want.abs() + 2.0 ** -17 * mag)
    cols = slice(H - 16, H)
    want = dout[:, cols].double().sum(0)
    R.check(db[cols], want, (T / 128 + 224) * 2.0 ** -24 * dout[:, cols].double().abs().sum(0))


def test_nothing_without_tokens(moe):
    torch = torch_()
    cfg = moe.make_config(128, 4, 2, 128, 8)
    ws = moe.workspace_grouped(cfg, 4)
    rows = moe.moe_max_padded_rows(cfg, 0)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    ids, counts = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    dw, add = torch.full((4, 16, 8), 7.0, device="cuda"), torch.randn(4, 16, 8, device="cuda")
    x, dy = torch.empty(0, 16, **bf), torch.empty(rows, 8, **bf)
    moe.moe_grouped_wgrad(cfg, 0, x, dy, ids, counts, dw, ws, dw_add=add, gather_x=True)
    assert torch.equal(dw, add)
    moe.moe_grouped_wgrad(cfg, 0, x, dy, ids, counts, dw, ws, gather_x=True)
    assert (dw == 0).all()
    moe.moe_grouped_gemm(cfg, 0, x, torch.empty(4, 16, 8, **bf), ids, counts, dy, ws, gather=True)
    v, w = torch.empty(0, 64, **bf), torch.ones(64, **bf)
    gw, gb = torch.full((64,), 7.0, device="cuda"), torch.full((64,), 7.0, device="cuda")
    moe.moe_norm_backward(v, v, None, w, 1e-5, v, gw, gb, moe.workspace_norm_backward(1, 64))
    assert (gw == 0).all() and (gb == 0).all()
    moe.moe_add_layer_norm(v, None, w, None, 1e-5, None, v)


@pytest.mark.parametrize("n", [768, 769, 1537, 9000, 30_001])
@pytest.mark.parametrize("add", [False, True])
def test_long_segments_keep_fp32_sums(moe, n, add):
    """A part of a long segment takes 48 MMA steps at most, each truncated by less than 2^-23 of the sum so far, and the
    parts are added rounded: 48 of 2^-23, however long the segment (without parts 30000 rows are 4e-5 to 8e-5 off)."""
    torch = torch_()
    N, K, F = 2, 264, 520
    cfg = moe.make_config(128, N, 1, 128, 8)
    g = _gen(n)
    counts = torch.tensor([n, 3], dtype=torch.int32, device="cuda")
    T = n + 3
    rows = moe.moe_max_padded_rows(cfg, T)
    ids = torch.full((rows,), T, dtype=torch.int32, device="cuda")
    start = (n + 7) // 8 * 8
    ids[:n], ids[start:start + 3] = torch.arange(n, device="cuda"), n + torch.arange(3, device="cuda")
    x = (torch.randn(T, K, generator=g, device="cuda") + 1).bfloat16()
    dy = torch.full((rows, F), float("nan"), dtype=torch.bfloat16, device="cuda")
    dy[:n], dy[start:start + 3] = (torch.randn(n, F, generator=g, device="cuda") + 1).bfloat16(), 1
    extra = torch.randn(N, K, F, generator=g, device="cuda") if add else None
    dw, ws = torch.empty(N, K, F, device="cuda"), moe.workspace_grouped(cfg, T)
    moe.moe_grouped_wgrad(cfg, T, x, dy, ids, counts, dw, ws, dw_add=extra, gather_x=True)
    half = torch.empty(N, K, F, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_wgrad(cfg, T, x, dy, ids, counts, half, ws, gather_x=True)
    assert moe.moe_get_device_status(ws) == 0
    want = torch.stack([x[:n].double().t() @ dy[:n].double(), x[n:].double().t() @ dy[start:start + 3].double()])
    got = dw.double() - (extra.double() if add else 0)
    assert float((got[0] - want[0]).norm() / want[0].norm()) <= 48 * 2.0 ** -23 + (2.0 ** -23 if add else 0)
    assert float((got[1] - want[1]).norm() / want[1].norm()) <= 4 * 2.0 ** -23 + (2.0 ** -23 if add else 0)
    # a bf16 gradient is rounded once; its parts are 512 steps long
    assert float((half[0].double() - want[0]).norm() / want[0].norm()) <= 2.0 ** -8 + 512 * 2.0 ** -23


@pytest.mark.parametrize("F", [2048, 2056, 1800])
@pytest.mark.parametrize("transposed", [False, True])
def test_one_and_two_groups_of_features_give_the_same_bits(moe, transposed, F):
    """4000 tokens, 2 of 4 experts, F about 2048: items of two groups where F fills them, of one where it does not."""
    torch = torch_()
    from tests import train_ref as R
    G, K, g = R.Groups(4000, 4, 2, 8, seed=5), 136, _gen(F)
    x, w = _randn(g, G.T, K), _randn(g, *((4, F, K) if transposed else (4, K, F)), scale=0.1)
    xp = torch.full((G.rows, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    xp[G.real] = x[G.ids[G.real].long() // G.k]
    y, yp = _gemm(moe, G, x, w, True, transposed), _gemm(moe, G, xp, w, False, transposed)
    assert torch.equal(y, yp)
    want, mag = R.gemm(G, x, w, True, transposed)
    R.check(y[G.real], want[G.real], R.BF * want[G.real].abs() + R.sum_tol(K) * mag[G.real])


def _at_16(t):
    """The same tensor at an address that is a multiple of 16, not of 32."""
    torch = torch_()
    step = 16 // t.element_size()
    flat = torch.empty(t.numel() + 2 * step, dtype=t.dtype, device="cuda")
    at = next(i for i in (step, 2 * step) if (flat.data_ptr() + i * t.element_size()) % 32 == 16)
    out = flat[at:at + t.numel()].view(t.shape)
    assert out.data_ptr() % 32 == 16
    return out.copy_(t)


def test_addresses_aligned_to_16_bytes_only(moe):
    torch = torch_()
    from tests import train_ref as R
    G, K, F, g = R.Groups(300, 5, 2, 8, seed=1, idle=(2,)), 200, 272, _gen(8)
    x, dy, w = _randn(g, G.T, K), G.grouped(F, g), _randn(g, 5, K, F)
    cfg, add = moe.make_config(128, 5, 2, 128, 8), torch.randn(5, K, F, generator=g, device="cuda")
    ws = moe.workspace_grouped(cfg, G.T)
    y = _gemm(moe, G, x, w, True, False)
    got = _at_16(torch.full_like(y, 7.0))
    moe.moe_grouped_gemm(cfg, G.T, _at_16(x), _at_16(w), _at_16(G.ids), _at_16(G.dcounts), got, ws, gather=True)
    assert torch.equal(got, y)
    for dtype, a in ((torch.float32, None), (torch.float32, add), (torch.bfloat16, None)):
        dw = torch.empty(5, K, F, dtype=dtype, device="cuda")
        moe.moe_grouped_wgrad(cfg, G.T, x, dy, G.ids, G.dcounts, dw, ws, dw_add=a, gather_x=True)
        got = _at_16(torch.full_like(dw, 7.0))
        moe.moe_grouped_wgrad(cfg, G.T, _at_16(x), _at_16(dy), _at_16(G.ids), G.dcounts, got, ws,
                              dw_add=None if a is None else _at_16(a), gather_x=True)
        assert torch.equal(got, dw)
    v, d, nw = _randn(g, 300, 272), _randn(g, 300, 272), _randn(g, 272)
    ref, out = torch.empty_like(v), _at_16(v)
    moe.moe_add_layer_norm(v, d, nw, None, 1e-5, None, ref)
    moe.moe_add_layer_norm(_at_16(v), _at_16(d), _at_16(nw), None, 1e-5, None, out)
    assert torch.equal(out, ref)
    nws = moe.workspace_norm_backward(300, 272)
    sums = torch.empty(2, 272, device="cuda")
    moe.moe_norm_backward(v, d, None, nw, 1e-5, ref, sums[0], sums[1], nws)
    odd = _at_16(torch.zeros_like(sums))
    moe.moe_norm_backward(_at_16(v), _at_16(d), None, _at_16(nw), 1e-5, out, odd[0], odd[1], nws)
    assert torch.equal(out, ref) and torch.equal(odd, sums)


def test_two_streams_share_a_grouped_workspace(moe):
    torch = torch_()
    from tests import train_ref as R
    G, K, F, g = R.Groups(2000, 6, 2, 16, seed=3), 512, 1024, _gen(4)
    x, dy, w = _randn(g, G.T, K), G.grouped(F, g), _randn(g, 6, K, F, scale=0.1)
    cfg = moe.make_config(128, 6, 2, 128, 16)
    ws = moe.workspace_grouped(cfg, G.T)
    want_y, want = _gemm(moe, G, x, w, True, False), torch.empty(6, K, F, device="cuda")
    moe.moe_grouped_wgrad(cfg, G.T, x, dy, G.ids, G.dcounts, want, ws, gather_x=True)
    y, dw = torch.full_like(want_y, 7.0), torch.empty_like(want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        y.fill_(7.0), dw.zero_()
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        moe.moe_grouped_gemm(cfg, G.T, x, w, G.ids, G.dcounts, y, ws, gather=True, stream=streams[0])
        moe.moe_grouped_wgrad(cfg, G.T, x, dy, G.ids, G.dcounts, dw, ws, gather_x=True, stream=streams[1])
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(dw, want)
    assert moe.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("transposed", [False, True])
def test_two_groups_gathered_and_one_in_place_give_the_same_bits(moe, transposed):
    """8192 rows of 8 experts, 56 groups of features: about 2016 tiles, for 76 pairs of CTAs 27 waves of single items or 14
    of double ones, which the gathered form takes (28 x 0.94 < 27) and the form in place does not (28 x 0.98 > 27)."""
    torch = torch_()
    from tests import train_ref as R
    G, K, F, g = R.Groups(4096, 8, 2, 8, seed=6), 72, 14336, _gen(6)
    x, w = _randn(g, G.T, K), _randn(g, *((8, F, K) if transposed else (8, K, F)), scale=0.1)
    xp = torch.full((G.rows, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    xp[G.real] = x[G.ids[G.real].long() // G.k]
    y, yp = _gemm(moe, G, x, w, True, transposed), _gemm(moe, G, xp, w, False, transposed)
    assert torch.equal(y, yp)


@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 96, 97, 127, 128, 129, 160, 161, 191, 192, 193,
                               224, 225, 255, 256, 257, 288, 289, 300, 352, 385, 480, 511, 512, 513, 545, 769])
def test_every_height_of_a_tile(moe, n):
    """An expert's rows in tiles of one height, followed by another expert's: in place (overlapping boxes, NaN in the padding)
    and gathered the same bits, both by the formula, nothing written past the segments."""
    torch = torch_()
    from tests import train_ref as R
    K, F, N, T = 200, 264, 2, n + 5
    g = _gen(n)
    cfg = moe.make_config(128, N, 1, 128, 8)
    rows = moe.moe_max_padded_rows(cfg, T)
    start = (n + 7) // 8 * 8
    real = torch.zeros(rows, dtype=torch.bool, device="cuda")
    real[:n] = real[start:start + 5] = True
    ids = torch.full((rows,), T, dtype=torch.int32, device="cuda")
    ids[real] = torch.randperm(T, generator=g, device="cuda").int()
    counts = torch.tensor([n, 5], dtype=torch.int32, device="cuda")
    x, w = _randn(g, T, K), _randn(g, N, K, F, scale=0.1)
    xp = torch.full((rows, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    xp[real] = x[ids[real].long()]
    ws = moe.workspace_grouped(cfg, T)
    ys = [torch.full((rows, F), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    moe.moe_grouped_gemm(cfg, T, x, w, ids, counts, ys[0], ws, gather=True)
    moe.moe_grouped_gemm(cfg, T, xp, w, None, counts, ys[1], ws)
    moe.moe_grouped_gemm(cfg, T, xp, w.transpose(1, 2).contiguous(), None, counts, ys[2], ws, transposed=True)
    assert moe.moe_get_device_status(ws) == 0
    a, b = xp[:n].double(), xp[start:start + 5].double()
    want = torch.cat([a @ w[0].double(), b @ w[1].double()])
    mag = torch.cat([a.abs() @ w[0].double().abs(), b.abs() @ w[1].double().abs()])
    assert torch.equal(ys[0], ys[1])
    for y in ys:
        assert (y[~real] == 7).all()
        R.check(y[real], want, R.BF * want.abs() + R.sum_tol(K) * mag)


@pytest.mark.parametrize("T,H", [(1, 8200), (400, 12288), (310, 12296), (333, 16384), (153, 10240), (1000, 8968)])
@pytest.mark.parametrize("centre", [True, False])
def test_norm_backward_of_wide_rows(moe, T, H, centre):
    test_norm_backward(moe, T, H, centre, 30.0)
