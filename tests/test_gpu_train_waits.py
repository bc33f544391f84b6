"""Bounded waits of the grouped products that run out: the status word reports it, nothing hangs, the next call is whole."""
import pytest

from tests.test_gpu_mx import moe, torch_  # noqa: F401
from tests.test_gpu_train import _gen, _randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,F", [(64, 128, 512), (700, 1096, 1032), (8000, 136, 2048)])
@pytest.mark.parametrize("form", ["in place", "gather", "transposed", "wgrad", "wgrad gather"])
def test_wait_runs_out_and_reports(moe, form, T, K, F):
    torch = torch_()
    from tests import train_ref as R
    N, k, B = 8, 2, 16
    G = R.Groups(T, N, k, B, skew=0.4, idle=(3,))
    g = _gen(1)
    out = {}
    for limit in (0, 1, 20000, 1, 0):   # none, 1 ns, 20 us
        cfg = moe.make_config(128, N, k, 128, B, debug_wait_ns=limit)
        ws = moe.workspace_grouped(cfg, T)
        g.manual_seed(1)
        if form.startswith("wgrad"):
            gx = form.endswith("gather")
            x, dy = (_randn(g, T, K) if gx else G.grouped(K, g)), G.grouped(F, g)
            y = torch.zeros(N, K, F, device="cuda")
            moe.moe_grouped_wgrad(cfg, T, x, dy, G.ids, G.dcounts, y, ws, gather_x=gx)
        else:
            gather, tr = form == "gather", form == "transposed"
            x = _randn(g, T, K) if gather else G.grouped(K, g)
            w = _randn(g, *((N, F, K) if tr else (N, K, F)))
            y = torch.zeros(G.rows, F, dtype=torch.bfloat16, device="cuda")
            moe.moe_grouped_gemm(cfg, T, x, w, G.ids, G.dcounts, y, ws, gather=gather, transposed=tr)
        torch.cuda.synchronize()
        status = moe.moe_get_device_status(ws)
        if limit == 1:
            assert status == moe.MOE_DEV_ERR_TIMEOUT
        elif limit == 0:
            assert status == 0
            assert torch.equal(out.setdefault("y", y), y)
        else:
            assert status in (0, moe.MOE_DEV_ERR_TIMEOUT)
