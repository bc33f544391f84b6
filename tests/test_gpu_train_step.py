"""The whole training step of a pre-norm MoE layer: a forward that keeps what its gradient needs, and the gradient,
through the public entry points, against 64-bit autograd; captured into a graph, on another stream, with capacity."""
import pytest

from tests.test_gpu_mx import moe, torch_  # noqa: F401
from tests.test_gpu_train import _gen, _randn

pytestmark = pytest.mark.gpu
EPS = 1e-5


class Step:
    def __init__(self, moe, T, H, N, k, I, B, seed=0, **cfg):
        torch = torch_()
        g = _gen(seed)
        self.moe, self.T, self.H, self.N, self.I = moe, T, H, N, I
        self.cfg = c = moe.make_config(H, N, k, I, B, **cfg)
        self.S = N if cfg.get("routing") else k
        self.x, self.r, self.dout = _randn(g, T, H), _randn(g, T, H), _randn(g, T, H)
        self.nw = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).bfloat16()
        self.nb = _randn(g, H, scale=0.1)
        self.wg, self.w13, self.w2 = (_randn(g, *s, scale=s[-2] ** -0.5) for s in ((H, N), (N, H, 2 * I), (N, I, H)))
        self.ws, self.gws = moe.workspace(c, T), moe.workspace_grouped(c, T)
        moe.moe_clear_device_status(self.ws)
        self.nws = moe.workspace_norm_backward(T, H)
        rows = self.rows = moe.moe_max_padded_rows(c, T)
        bf, i32, f32 = (dict(dtype=d, device="cuda") for d in (torch.bfloat16, torch.int32, torch.float32))
        nan = float("nan")
        self.v, self.n, self.out, self.dn, self.dx = (torch.empty(T, H, **bf) for _ in range(5))
        self.gu, self.dgu = (torch.full((rows, 2 * I), nan, **bf) for _ in range(2))
        self.a, self.a2, self.da = (torch.full((rows, I), nan, **bf) for _ in range(3))
        self.y, self.dxp = (torch.full((rows, H), nan, **bf) for _ in range(2))
        self.idx, self.gate = torch.empty(T, k, **i32), torch.empty(T, self.S, **f32)
        self.logits = torch.empty(T, N, **f32)
        self.dgate = torch.zeros(T, self.S, **f32)
        self.kept, self.pos = torch.empty(T * self.S, dtype=torch.uint8, device="cuda"), torch.empty(T * self.S, **i32)
        self.ids, self.blocks = torch.empty(rows, **i32), torch.empty(moe.moe_max_blocks(c, T), **i32)
        self.npad, self.counts, self.dropped = torch.zeros(1, **i32), torch.empty(N, **i32), torch.empty(1, **i32)
        self.ones = torch.ones(T, self.S, **f32)
        self.dw13, self.dw2 = torch.zeros(N, H, 2 * I, **f32), torch.empty(N, I, H, **bf)
        self.dnw, self.dnb = torch.empty(H, **f32), torch.empty(H, **f32)

    def route(self):
        m, c = self.moe, self.cfg
        m.moe_add_layer_norm(self.x, self.r, self.nw, self.nb, EPS, self.v, self.n)
        if c.routing:
            m.moe_router_logits(c, self.n, self.wg, None, self.logits, self.ws)
            m.moe_route_expert_choice(c, self.logits, self.gate, self.kept, self.pos, self.ids, self.blocks, self.npad,
                                      self.counts, self.ws)
        else:
            m.moe_route(c, self.n, self.wg, None, self.idx, self.gate, None, self.ws)
            m.moe_dispatch_align(c, self.idx, self.kept, self.pos, self.ids, self.blocks, self.npad, self.counts,
                                 self.dropped, self.ws)

    def forward(self):
        m, c, T = self.moe, self.cfg, self.T
        m.moe_grouped_gemm(c, T, self.n, self.w13, self.ids, self.counts, self.gu, self.gws, gather=True)
        m.moe_swiglu(c, T, self.gu, self.gate, self.ids, self.npad, self.a)
        m.moe_grouped_gemm(c, T, self.a, self.w2, None, self.counts, self.y, self.gws)
        m.moe_combine(c, self.v, self.ones, self.kept, self.pos, self.y, None, self.out)

    def backward(self):
        m, c, T = self.moe, self.cfg, self.T
        m.moe_grouped_gemm(c, T, self.dout, self.w2, self.ids, self.counts, self.da, self.gws, gather=True, transposed=True)
        m.moe_swiglu_backward(c, T, self.gu, self.gate, self.da, self.ids, self.npad, self.dgu, self.dgate, self.a2)
        m.moe_grouped_wgrad(c, T, self.a2, self.dout, self.ids, self.counts, self.dw2, self.gws, gather_dy=True)
        m.moe_grouped_wgrad(c, T, self.n, self.dgu, self.ids, self.counts, self.dw13, self.gws, dw_add=self.dw13,
                            gather_x=True)
        m.moe_grouped_gemm(c, T, self.dgu, self.w13, None, self.counts, self.dxp, self.gws, transposed=True)
        # the rows' gradients sum into the norm's output's; the combine's residual is zero there
        m.moe_combine(c, self.zero(), self.ones, self.kept, self.pos, self.dxp, None, self.dn)
        m.moe_norm_backward(self.v, self.dn, self.dout, self.nw, EPS, self.dx, self.dnw, self.dnb, self.nws)

    def zero(self):
        if not hasattr(self, "_zero"):
            self._zero = torch_().zeros_like(self.dout)
        return self._zero

    def results(self):
        return {n: getattr(self, n) for n in ("out", "dx", "dw13", "dw2", "dgate", "dnw", "dnb")}

    def reference(self):
        """Autograd in 64 bits over the same routes; the gates are leaves, as the router's gradient is the caller's."""
        torch = torch_()
        from tests import train_ref as R
        x, r, nw, nb, w13, w2, gate = (t.double().requires_grad_() for t in (self.x, self.r, self.nw, self.nb, self.w13,
                                                                            self.w2, self.gate))
        v = x + r
        n = R.layer_norm(v, nw, nb, EPS)
        out = v
        starts, at = [], 0
        for c in self.counts.tolist():
            starts.append((at, c))
            at += -(-c // self.cfg.block_size) * self.cfg.block_size
        for e, (p, c) in enumerate(starts):
            route = self.ids[p:p + c].long()
            t = route // self.S
            g, u = (n[t] @ w13[e]).split(self.I, -1)
            out = out.index_add(0, t, R.swiglu(g, u, gate.flatten()[route].unsqueeze(-1)) @ w2[e])
        out.backward(self.dout.double())
        assert torch.equal(x.grad, r.grad)
        return dict(out=out.detach(), dx=x.grad, dw13=w13.grad, dw2=w2.grad, dgate=gate.grad, dnw=nw.grad, dnb=nb.grad)


CASES = [dict(T=64, H=128, N=8, k=2, I=256, B=8), dict(T=1, H=256, N=16, k=4, I=128, B=128),
         dict(T=500, H=384, N=12, k=3, I=640, B=16), dict(T=300, H=256, N=6, k=2, I=384, B=32, capacity_factor=0.7),
         dict(T=200, H=256, N=5, k=2, I=256, B=8, routing=1)]


@pytest.mark.parametrize("case", CASES)
def test_step_against_autograd(moe, case):
    torch = torch_()
    s = Step(moe, seed=case["T"], **case)
    s.route()
    s.forward()
    s.backward()
    assert moe.moe_get_device_status(s.ws) == 0 and moe.moe_get_device_status(s.gws) == 0
    if "capacity_factor" in case:
        assert int(s.dropped) > 0
    for name, want in s.reference().items():
        got = s.results()[name].double()
        assert torch.isfinite(got).all()
        # eight bf16 roundings on the longest path (gu, a, y, out, da, dgu, dx, dn), each 2^-8 of its value at most; the
        # products of random matrices keep relative sizes, the activation's slope at most doubles them
        err = float((got - want).norm() / want.norm())
        assert err <= 8 * 2 * 2.0 ** -8, (name, err)
    # the same outputs again, on another stream and replayed from a graph; dw13 is added to, so it starts from zero
    first = {n: t.clone() for n, t in s.results().items()}

    def again():
        for t in s.results().values():
            t.zero_()
        s.route()
        s.forward()
        s.backward()

    def same():
        torch.cuda.synchronize()
        assert all(torch.equal(first[n], t) for n, t in s.results().items())
    s.zero()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again()
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again()
    for t in s.results().values():
        t.fill_(3)
    graph.replay()
    same()


def test_two_graphs_share_a_workspace(moe):
    torch = torch_()
    steps = [Step(moe, seed=1, **CASES[0]), Step(moe, seed=2, **CASES[2])]
    want, graphs = [], []
    big = steps[1]
    for s in steps:   # one workspace of each kind for both
        s.ws, s.gws, s.nws = big.ws, big.gws, big.nws
        s.zero()
        s.route(), s.forward(), s.backward()
        want.append({n: t.clone() for n, t in s.results().items() if n != "dw13"})
    torch.cuda.synchronize()
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.route(), s.forward(), s.backward()
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, getattr(steps[i], n)) for n, t in want[i].items())


def test_accumulation_over_batches(moe):
    """dw_add sums the gradients of several batches: the bits of the two calls in turn."""
    torch = torch_()
    s = Step(moe, seed=4, **CASES[0])
    s.route(), s.forward(), s.backward()
    one = s.dw13.clone()
    s.backward()
    fresh = torch.empty_like(one)
    moe.moe_grouped_wgrad(s.cfg, s.T, s.n, s.dgu, s.ids, s.counts, fresh, s.gws, dw_add=one, gather_x=True)
    assert torch.equal(fresh, s.dw13) and (fresh - 2 * one).abs().max() <= 2.0 ** -22 * one.abs().max()
