"""moe_route_scored at the ends of the score range."""
import numpy as np
import pytest

from tests import mx_ref
from tests.test_gpu_mx import _route, moe  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,groups,top_groups", [(256, 8, 4), (128, 1, 1), (32, 2, 1), (60, 5, 3), (7, 1, 1)])
def test_subnormal_sigmoid_scores_rank(moe, N, groups, top_groups):
    """1 / (1 + exp(-l)) between l = -88.7 and -87.3 is subnormal, not 0."""
    rng = np.random.default_rng(N)
    # distinct scores, 1 part in 300 apart at least (a subnormal score has 20 bits here)
    l = np.stack([rng.permutation(np.linspace(-88.6, -87.4, N)) for _ in range(40)]).astype(np.float32)
    k = min(4, top_groups * (N // groups))
    idx, gate, margin = mx_ref.route(l, None, k, True, groups, top_groups)
    assert (margin > 1e-42).all()
    got_idx, got_gate = _route(moe, l, None, k, True, groups, top_groups, False, False)
    np.testing.assert_array_equal(got_idx, idx)
    # exponential and reciprocal in fp32, and half a unit of a subnormal number
    np.testing.assert_allclose(got_gate, gate, rtol=2e-6, atol=2.0 ** -149)
    # past the fp32 exponential every score is 0: the lower index
    got_idx, got_gate = _route(moe, l - 2, None, k, True, groups, top_groups, False, False)
    assert (got_idx == np.arange(k)).all() and (got_gate == 0).all()


@pytest.mark.parametrize("N,groups,top_groups,top2", [(256, 8, 4, True), (128, 4, 2, False), (128, 1, 1, False), (64, 16, 5, True),
                                                      (96, 3, 2, True)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("closed", [1, 0.3, 0.9, "group", "all"])
def test_experts_closed_by_the_bias(moe, N, groups, top_groups, top2, sigmoid, closed):
    """score_bias -inf: never chosen while k others are left in the groups that stay, and then by index."""
    rng = np.random.default_rng(N + groups)
    l = rng.standard_normal((133, N)).astype(np.float32)
    bias = 0.05 * rng.standard_normal(N)
    size = N // groups
    if closed == "group":
        bias[size * (groups // 2):size * (groups // 2 + 1)] = -np.inf
    elif closed == "all":
        bias[:] = -np.inf
    else:
        bias[rng.permutation(N)[:max(1, int(closed * N) if closed < 1 else 1)]] = -np.inf
    bias = bias.astype(np.float32)
    k = min(6, top_groups * size)
    l[5, 3], l[7, 2], l[9] = np.nan, np.inf, -np.inf        # and odd logits beside them
    rows = np.arange(len(l)) if sigmoid else np.setdiff1d(np.arange(len(l)), [5, 7])
    with np.errstate(invalid="ignore"):
        idx, gate, margin = mx_ref.route(l[rows], bias, k, sigmoid, groups, top_groups, top2, True)
    # ties of equal scores (rows of -inf) and of closed experts are exact; others are kept apart
    keep = ~(margin < 2e-6) | (margin == 0)
    assert keep.sum() > 100
    got_idx, got_gate = _route(moe, l, bias, k, sigmoid, groups, top_groups, top2, True)
    np.testing.assert_array_equal(got_idx[rows][keep], idx[keep])
    np.testing.assert_allclose(got_gate[rows][keep], gate[keep], rtol=2e-6, atol=1e-12)
