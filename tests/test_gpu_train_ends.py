"""The training step's operators at the ends of their values: NaN and infinities in an operand's row stay where the formula
puts them, and eps = 0."""
import pytest

from tests.test_gpu_mx import moe, torch_  # noqa: F401
from tests.test_gpu_train import _gemm, _gen, _randn

pytestmark = pytest.mark.gpu


# tokens, experts, choices, columns: items of one group of features, and of two
@pytest.mark.parametrize("T,N,k,K,F", [(300, 5, 2, 200, 272), (4000, 4, 2, 136, 2048)])
@pytest.mark.parametrize("transposed", [False, True])
def test_products_keep_nan_and_infinities_in_their_rows(moe, T, N, k, K, F, transposed):
    torch = torch_()
    from tests import train_ref as R
    G, g = R.Groups(T, N, k, 8, seed=1), _gen(K)
    x, w = _randn(g, T, K), _randn(g, *((N, F, K) if transposed else (N, K, F)))
    bad = x.clone()
    bad[T // 3, 7], bad[T // 2, K - 1], bad[T - 1, 0] = float("nan"), float("inf"), -float("inf")
    token = G.ids[G.real].long() // k
    for gather in (True, False):
        ys = []
        for v in (x, bad):
            if not gather:
                grouped = torch.full((G.rows, K), float("nan"), dtype=torch.bfloat16, device="cuda")
                grouped[G.real] = v[token]
                v = grouped
            ys.append(_gemm(moe, G, v, w, gather, transposed)[G.real])
        hit = (token == T // 3) | (token == T // 2) | (token == T - 1)
        assert int(hit.sum()) == 3 * k
        assert torch.equal(ys[0][~hit], ys[1][~hit]) and not torch.isfinite(ys[1][hit]).any()


@pytest.mark.parametrize("add", [False, True])
def test_weight_gradients_keep_nan_and_infinities_in_their_columns(moe, add):
    torch = torch_()
    from tests import train_ref as R
    T, N, k, K, F = 3000, 3, 1, 200, 272      # segments of some 1000 rows: two parts
    G, g = R.Groups(T, N, k, 8, seed=2), _gen(3)
    x, dy = _randn(g, T, K), G.grouped(F, g)
    extra = torch.randn(N, K, F, generator=g, device="cuda") if add else None
    cfg = moe.make_config(128, N, k, 128, 8)
    ws = moe.workspace_grouped(cfg, T)

    def grad(x, dy):
        dw = torch.empty(N, K, F, device="cuda")
        moe.moe_grouped_wgrad(cfg, T, x, dy, G.ids, G.dcounts, dw, ws, dw_add=extra, gather_x=True)
        return dw
    clean = grad(x, dy)
    bx, bdy = x.clone(), dy.clone()
    p = G.start[2] + G.counts[2] - 1
    bdy[p, 3] = float("inf")                       # the last row of expert 2
    r = G.start[1] + 5
    bx[G.ids[r].long(), 7] = float("nan")          # a row of expert 1
    dw = grad(bx, bdy)
    hit = torch.zeros(N, K, F, dtype=torch.bool, device="cuda")
    hit[1, 7], hit[2, :, 3] = True, True
    assert torch.equal(dw[~hit], clean[~hit]) and not torch.isfinite(dw[hit]).any()


def test_silu_of_every_bf16_value(moe):
    """dgate of rows with one element whose da and u are 1 is silu(g) itself.  The exponential is off by (2 + 1.173 |g|) 2^-23,
    the division by 2^-22 and the addition and the product with g by 2^-24 each: within (6 + 1.2 |g|) 2^-23."""
    torch = torch_()
    from tests import train_ref as R
    bits = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    G = R.Groups(v.numel(), 1, 1, 8)
    gu, da = (torch.zeros(G.rows, n, dtype=torch.bfloat16, device="cuda") for n in (256, 128))
    token = G.ids[G.real].long()
    gu[G.real, 5], gu[:, 128 + 5], da[:, 5] = v[token], 1, 1
    dgu, dgate = torch.empty_like(gu), torch.empty(v.numel(), 1, device="cuda")
    cfg = moe.make_config(128, 1, 1, 128, 8)
    moe.moe_swiglu_backward(cfg, v.numel(), gu, None, da, G.ids, G.num_padded, dgu, dgate)
    g, got = v.double(), dgate.flatten().double()
    want = g * torch.sigmoid(g)
    near = g >= -87.3
    # (results below 2^-126 have no 24 bits)
    R.check(got[near], want[near], (6 + 1.2 * g[near].abs().clamp(max=200)) * 2.0 ** -23 * want[near].abs() + 2.0 ** -149)
    assert (got[g < -87.4] == 0).all() and want[g < -87.3].abs().max() < 2.0 ** -119


WIDTHS = [264, 4096, 7168, 12288, 16392]           # a form of the norms each


@pytest.mark.parametrize("H", WIDTHS)
def test_layer_norm_keeps_nan_and_infinities_in_their_rows(moe, H):
    torch = torch_()
    T, g = 700, _gen(H)
    x, r, w, b = _randn(g, T, H), _randn(g, T, H), _randn(g, H), _randn(g, H)
    bad = x.clone()
    bad[5, 3], bad[7, H - 1], bad[698, 0] = float("nan"), float("inf"), -float("inf")
    rows = [5, 7, 698]
    got = []
    for v in (x, bad):
        out, v_out = torch.empty_like(v), torch.empty_like(v)
        moe.moe_add_layer_norm(v, r, w, b, 1e-5, v_out, out)
        got.append((out, v_out))
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert torch.isnan(got[1][0][rows]).all() and torch.equal(got[0][0][rest], got[1][0][rest])
    same = torch.equal(torch.isnan(bad), torch.isnan(got[1][1])) and torch.equal(torch.isinf(bad), torch.isinf(got[1][1]))
    assert same and torch.equal(got[0][1][torch.isfinite(bad)], got[1][1][torch.isfinite(bad)])


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("centre", [True, False])
def test_norm_backward_keeps_nan_and_infinities_where_they_belong(moe, H, centre):
    torch = torch_()
    T, g = 700, _gen(H)
    v, d, w = _randn(g, T, H), _randn(g, T, H), _randn(g, H)
    ws = moe.workspace_norm_backward(T, H)

    def grad(v, d):
        dx, dw, db = torch.empty_like(v), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
        moe.moe_norm_backward(v, d, None, w, 1e-5, dx, dw, db, ws, centre=centre)
        return dx, dw, db
    dx, dw, db = grad(v, d)
    rest, cols = torch.ones(T, dtype=torch.bool, device="cuda"), torch.ones(H, dtype=torch.bool, device="cuda")
    rest[[5, 699]], cols[3] = False, False
    # in the incoming gradient: the row of dx, and the column of both sums
    bad = d.clone()
    bad[5, 3], bad[699, 3] = float("nan"), float("inf")
    bx, bw, bb = grad(v, bad)
    # (an infinite mean(g) and mean(g n) leave inf - inf or inf + inf, by their signs)
    assert torch.equal(bx[rest], dx[rest]) and torch.isnan(bx[5]).all() and not torch.isfinite(bx[699]).any()
    for s, clean in ((bw, dw), (bb, db)):
        assert torch.equal(s[cols], clean[cols]) and torch.isnan(s[3])
    # in the normalised row: its dx, all of dweight, nothing of dbias
    bad = v.clone()
    bad[5, 3], bad[699, 0] = float("nan"), float("nan")
    bx, bw, bb = grad(bad, d)
    assert torch.equal(bx[rest], dx[rest]) and torch.isnan(bx[~rest]).all()
    assert torch.isnan(bw).all() and torch.equal(bb, db)


@pytest.mark.parametrize("H", [1024, 4096, 16384, 32768])
def test_norms_without_eps(moe, H):
    """Rows of equal values whose sum is exact (H is a power of two) have no deviation: NaN with eps = 0, in their row of the
    forward and of dx and in all of dweight, and in nothing else.  Other rows are normalised as with any eps."""
    torch = torch_()
    from tests import train_ref as R
    T, g = 40, _gen(H)
    x, d, w, b = _randn(g, T, H), _randn(g, T, H), _randn(g, H), _randn(g, H)
    clean = x.clone()
    x[3], x[17] = 1.5, 0.0
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[[3, 17]] = False
    out, ref = torch.empty_like(x), torch.empty_like(x)
    moe.moe_add_layer_norm(x, None, w, b, 0.0, None, out)
    moe.moe_add_layer_norm(clean, None, w, b, 0.0, None, ref)
    assert torch.isnan(out[~rest]).all() and torch.equal(out[rest], ref[rest])
    want = R.layer_norm(clean.double(), w.double(), b.double(), 0.0)
    n = (want - b.double()).abs()
    # the slack of test_add_layer_norm: 64 of 2^-24 of each term, and the mean's error in every deviation (root 1: unit normals)
    slack = 2.0 ** -18 * (n + b.double().abs() + 2 * clean.double().abs().mean(-1, keepdim=True) * w.double().abs())
    R.check(ref, want, R.BF * want.abs() + slack)
    ws = moe.workspace_norm_backward(T, H)
    for centre in (True, False):
        got = []
        for v in (x, clean):
            dx, dw, db = torch.empty_like(v), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
            moe.moe_norm_backward(v, d, None, w, 0.0, dx, dw, db, ws, centre=centre)
            got.append((dx, dw, db))
        gone = ~rest
        if not centre:   # the RMS norm of 1.5 is defined
            gone[3] = False
        assert torch.isnan(got[0][0][gone]).all() and torch.equal(got[0][0][rest], got[1][0][rest])
        assert torch.isfinite(got[0][0][~gone]).all() and torch.isfinite(got[1][1]).all()
        assert torch.isnan(got[0][1]).all() and torch.equal(got[0][2], got[1][2])
