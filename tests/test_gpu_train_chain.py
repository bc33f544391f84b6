"""Training steps queued one after another on the same buffers with other inputs each time: every launch may start while the
one before it ends, and reads the counts, route ids, gates and rows of its own step."""
import pytest

from tests.test_gpu_mx import moe, torch_  # noqa: F401
from tests.test_gpu_train import _gen, _randn
from tests.test_gpu_train_step import CASES, Step

pytestmark = pytest.mark.gpu

CHAINS = CASES + [dict(T=3000, H=512, N=32, k=4, I=384, B=16)]


@pytest.mark.parametrize("case", CHAINS)
def test_queued_steps_read_their_own_inputs(moe, case):
    torch = torch_()
    s = Step(moe, seed=case["T"], **case)
    s.zero()
    torch.cuda.synchronize()
    inputs = [(_randn(_gen(i), s.T, s.H), _randn(_gen(100 + i), s.T, s.H)) for i in range(5)]

    class EachCall:
        """The library with a wait behind every call."""
        def __getattr__(self, name):
            f = getattr(moe, name)

            def call(*a, **k):
                r = f(*a, **k)
                torch.cuda.synchronize()
                return r
            return call

    def step(i):
        s.x.copy_(inputs[i][0])
        s.dout.copy_(inputs[i][1])
        s.dw13.zero_()
        s.dgate.zero_()
        s.route(), s.forward(), s.backward()
        return {n: t.clone() for n, t in s.results().items()}
    s.moe = EachCall()
    want = [step(i) for i in range(5)]
    assert not torch.equal(want[0]["out"], want[1]["out"])
    s.moe = moe
    order = [0, 3, 1, 4, 2, 0, 2, 4, 1, 3] * 3
    got = [step(i) for i in order]
    torch.cuda.synchronize()
    for i, g in zip(order, got):
        assert all(torch.equal(want[i][n], g[n]) for n in g)
    assert moe.moe_get_device_status(s.ws) == 0 and moe.moe_get_device_status(s.gws) == 0
