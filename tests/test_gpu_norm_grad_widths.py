"""The norms' gradient at row widths between its forms (4096 and 8192 columns) against the formula in 64 bits."""
import pytest

from tests.test_gpu_mx import moe  # noqa: F401
from tests.test_gpu_train import test_norm_backward as check_norm_backward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(310, 4104), (310, 7176), (5, 7424), (310, 7680), (310, 7688), (153, 8192)])
@pytest.mark.parametrize("centre", [True, False])
def test_norm_backward_up_to_8192_columns(moe, T, H, centre):
    check_norm_backward(moe, T, H, centre, 30.0)
