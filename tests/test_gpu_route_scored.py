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
