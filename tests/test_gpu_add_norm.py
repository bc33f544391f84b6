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


@pytest.mark.parametrize("T", [5, 700])   # one and four chunks a warp
def test_squares_past_the_fp32_range(moe, T):
    """The fp32 formula where the sum of squares vanishes or is infinite: v / 0 and v / inf."""
    torch = torch_()
    H = 1056
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    x[1] = 1e-30
    x[1, 3], x[1, 4] = -1e-30, 0
    x[2] = 0
    x[3] = 3e38
    out = torch.empty_like(x)
    codes, scales = mx_buffers((T,), H)
    w = torch.full((H,), 2.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_add_norm(x, None, w, 0.0, None, out, codes, scales)
    v = x.float()
    root = torch.sqrt((v * v).mean(-1, keepdim=True))
    assert root[1] == 0 and torch.isinf(root[3])
    want = (v / root * 2.0).bfloat16()
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.nan_to_num(nan=0.5, posinf=7, neginf=-7), want.nan_to_num(nan=0.5, posinf=7, neginf=-7))
    assert (scales[1:3] == 255).all() and (scales[3] == 0).all()
    moe.moe_add_norm(x, None, w, 1e-6, None, out)
    assert (out[2] == 0).all() and (out[3] == 0).all() and torch.isfinite(out[1]).all()
