"""moe_add_norm in place, and at the ends of the fp32 range."""
import numpy as np
import pytest

from tests.test_gpu_mx import bf16, moe, mx_buffers, torch_  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(2, 96), (3, 4096), (700, 1056), (650, 8704)])   # one and four chunks a warp
@pytest.mark.parametrize("r_out_is,out_is", [("x", None), ("r", None), (None, "x"), (None, "r"), ("x", "r"), ("r", "x")])
def test_outputs_may_be_the_inputs(moe, T, H, r_out_is, out_is):
    torch = torch_()
    rng = np.random.default_rng(T + H)
    x, r, w = bf16(rng.standard_normal((T, H))), bf16(rng.standard_normal((T, H))), bf16(1 + 0.1 * rng.standard_normal(H))
    want = torch.empty_like(x), torch.empty_like(x)
    wc = mx_buffers((T,), H)
    moe.moe_add_norm(x, r, w, 1e-6, *want, *wc)
    at = {"x": x.clone(), "r": r.clone(), None: torch.empty_like(x)}
    spare = torch.empty_like(x)
    r_out, out = at[r_out_is], at[out_is] if out_is else spare
    codes = mx_buffers((T,), H)
    moe.moe_add_norm(at["x"], at["r"], w, 1e-6, r_out, out, *codes)
    assert torch.equal(r_out, want[0]) and torch.equal(out, want[1])
    assert torch.equal(codes[0], wc[0]) and torch.equal(codes[1], wc[1])
