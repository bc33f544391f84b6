"""Block lists of a caller's own: ids out of range between routes, and segments whose last block, last blocks or only
blocks hold no route.  Routed rows keep their bits, rows without a route before a segment's last one are zeros, and
rows past it are not written."""
import numpy as np
import pytest

from tests.gpu_util import host
from tests.test_gpu_mx import Layer, _tokens, moe, torch_  # noqa: F401

pytestmark = pytest.mark.gpu


def _blank(ids, blocks, P, B, R, rng):
    """ids with routes taken out: by expert in turn the last block, the last three, all, every block but the first's
    first row, scattered rows, and none.  Returns them and, per row, 'route', 'zero' or 'kept' (not written)."""
    ids = ids.copy()
    of = np.repeat(blocks[:P // B], B)
    state = np.full(len(ids), "kept", object)
    for e in np.unique(of):
        rows = np.flatnonzero(of == e)
        way = e % 6
        if way == 0:
            ids[rows[-B:]] = R
        elif way == 1:
            ids[rows[-3 * B:]] = R
        elif way == 2:
            ids[rows] = -7
        elif way == 3:
            ids[rows[1:]] = 2 ** 31 - 1
        elif way == 4:
            ids[rows[rng.random(len(rows)) < 0.4]] = R
            ids[rows[0]] = -1
        routes = rows[(ids[rows] >= 0) & (ids[rows] < R)]
        if routes.size:
            state[rows[rows < routes[-1]]] = "zero"
            state[routes] = "route"
    return ids, state


def _compare(y, want, state):
    got, want = host(y.float()), host(want.float())
    assert (got[state == "route"] == want[state == "route"]).all()
    assert (got[state == "zero"] == 0).all()
    assert (got[state == "kept"] == 7).all()
    assert min((state == s).sum() for s in ("route", "zero", "kept")) > 0


CASES = [  # T, N, k, B, form: blocks below, at and above the tile's height
    (40, 12, 2, 8, 32), (60, 12, 2, 32, 32), (60, 12, 2, 128, 32), (40, 8, 1, 64, 32),
    (200, 12, 2, 8, 128), (300, 12, 2, 128, 128),
    (1500, 12, 2, 8, 256), (1500, 12, 2, 64, 256), (900, 7, 2, 128, 256)]


@pytest.mark.parametrize("T,N,k,B,form", CASES)
def test_mx_ffn(moe, T, N, k, B, form):
    torch = torch_()
    L = Layer(moe, 256, N, k, 384, B, seed=T)
    assert moe.moe_expert_ffn_mx_tile_rows(L.cfg, T) == form
    rng = np.random.default_rng(T + B)
    c, s = (torch.from_numpy(v).cuda() for v in _tokens(rng, T, 256))
    idx = torch.from_numpy(np.sort(np.argsort(rng.random((T, N)), axis=1)[:, :k], axis=1).astype(np.int32)).cuda()
    d = L.dispatch(idx)
    want, _ = L.ffn(c, s, d)
    ids, state = _blank(host(d["ids"]), host(d["blocks"]), int(d["npad"][0]), B, T * k, rng)
    y, _ = L.ffn(c, s, dict(d, ids=torch.from_numpy(ids).cuda()))
    _compare(y, want, state)


@pytest.mark.parametrize("T,N,k,B", [(60, 12, 2, 8), (200, 12, 2, 128), (1500, 12, 2, 8)])
def test_bf16_ffn(moe, T, N, k, B):
    torch = torch_()
    rng = np.random.default_rng(T + B)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    H, I = 256, 384
    cfg = moe.make_config(H, N, k, I, B)
    h, w13, w2 = (torch.randn(*n, generator=g, device="cuda").mul_(f).bfloat16()
                  for n, f in (((T, H), 1.0), ((N, H, 2 * I), 0.05), ((N, I, H), 0.05)))
    e = dict(device="cuda", dtype=torch.int32)
    rows = moe.moe_max_padded_rows(cfg, T)
    ids, blocks, npad = torch.full((rows,), -9, **e), torch.full((moe.moe_max_blocks(cfg, T),), -9, **e), torch.zeros(1, **e)
    idx = torch.from_numpy(np.sort(np.argsort(rng.random((T, N)), axis=1)[:, :k], axis=1).astype(np.int32)).cuda()
    ws = moe.workspace(cfg, T)
    moe.moe_clear_device_status(ws)
    moe.moe_dispatch_align(cfg, idx, torch.empty(T * k, dtype=torch.uint8, device="cuda"), torch.empty(T * k, **e), ids, blocks,
                           npad, torch.empty(N, **e), torch.empty(1, **e), ws)

    def ffn(ids):
        y = torch.full((rows, H), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_expert_ffn(cfg, h, w13, w2, None, None, ids, blocks, npad, y, None, ws)
        assert moe.moe_get_device_status(ws) == 0
        return y
    want = ffn(ids)
    blank, state = _blank(host(ids), host(blocks), int(npad[0]), B, T * k, rng)
    _compare(ffn(torch.from_numpy(blank).cuda()), want, state)
