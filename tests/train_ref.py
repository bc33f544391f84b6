"""The training step's operators from their formulas in 64 bits, and layouts for their tests."""
import torch

BF = 2.0 ** -8      # half a step of bf16, relative
F64 = torch.float64


def swiglu(g, u, w):
    return w * (g * torch.sigmoid(g)) * u


def swiglu_backward(g, u, w, da):
    """(dg, du, dw): dw per row."""
    s = torch.sigmoid(g)
    return w * da * u * s * (1 + g * (1 - s)), w * da * g * s, (da * g * s * u).sum(-1)


def layer_norm(v, weight, bias, eps):
    d = v - v.mean(-1, keepdim=True)
    return d / torch.sqrt((d * d).mean(-1, keepdim=True) + eps) * weight + bias


def rms_norm(v, weight, eps):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * weight


def norm_backward(v, dout, dres, weight, eps, centre):
    """dx, dweight, dbias, and the magnitudes that errors of dx and dweight scale with."""
    H = v.shape[-1]
    mean_abs = v.abs().mean(-1, keepdim=True)
    d = v - v.mean(-1, keepdim=True) if centre else v
    inv = 1 / torch.sqrt((d * d).mean(-1, keepdim=True) + eps)
    n, g = d * inv, dout * weight
    mgn = (g * n).mean(-1, keepdim=True)
    dx = inv * (g - n * mgn - (g.mean(-1, keepdim=True) if centre else 0)) + dres
    mag_g, mag_gn = g.abs().mean(-1, keepdim=True), (g * n).abs().mean(-1, keepdim=True)
    mag = inv * (g.abs() + mag_g + n.abs() * mag_gn + inv * mean_abs * (mag_gn + n.abs() * mag_g)) + dres.abs()
    mag_w = (dout.abs() * (n.abs() + inv * mean_abs)).sum(0)
    assert dx.shape[-1] == H
    return dx, (dout * n).sum(0), dout.sum(0), mag, mag_w, dout.abs().sum(0)


class Groups:
    """Routes of T tokens to k of N experts each in moe_dispatch_align's layout.  skew: the share of tokens whose
    first choice is expert 0; idle experts take no route."""

    def __init__(self, T, N, k, B, seed=0, skew=0.0, idle=(), device="cuda"):
        g = torch.Generator().manual_seed(seed)
        score = torch.rand(T, N, generator=g)
        for e in idle:
            score[:, e] = -1
        if skew:
            score[torch.rand(T, generator=g) < skew, 0] = 2
        idx = score.topk(k, -1).indices.sort(-1).values
        assert not (set(idle) & set(idx.flatten().tolist()))
        flat = idx.flatten()
        self.T, self.N, self.k, self.B, self.R = T, N, k, B, T * k
        self.counts = torch.bincount(flat, minlength=N).tolist()
        self.start, at = [], 0
        self.rows = T * k + N * (B - 1)
        ids = torch.full((self.rows,), self.R, dtype=torch.int32)
        order = torch.argsort(flat, stable=True)
        first = 0
        for n in self.counts:
            self.start.append(at)
            ids[at:at + n] = order[first:first + n].int()
            first += n
            at += (n + B - 1) // B * B
        self.padded = at
        self.ids = ids.to(device)
        self.dcounts = torch.tensor(self.counts, dtype=torch.int32, device=device)
        self.num_padded = torch.tensor([at], dtype=torch.int32, device=device)
        self.real = ((ids >= 0) & (ids < self.R) & (torch.arange(self.rows) < at)).to(device)

    def token(self, p0, n):
        return self.ids[p0:p0 + n].long() // self.k

    def grouped(self, columns, g, fill=float("nan"), scale=1.0):
        """A grouped bf16 tensor: numbers where there is a row, `fill` elsewhere."""
        x = torch.randn(self.rows, columns, generator=g, device=self.ids.device).mul_(scale).bfloat16()
        x[~self.real] = fill
        return x


def gemm(G, x, w, gather, transposed):
    """y and the sums of the products' magnitudes, [rows, F] in 64 bits (zeros without a row)."""
    F = w.shape[1] if transposed else w.shape[2]
    y = torch.zeros(G.rows, F, dtype=F64, device=x.device)
    m = torch.zeros_like(y)
    for e, (p, n) in enumerate(zip(G.start, G.counts)):
        if n:
            rows = (x[G.token(p, n)] if gather else x[p:p + n]).double()
            we = w[e].double().t() if transposed else w[e].double()
            y[p:p + n], m[p:p + n] = rows @ we, rows.abs() @ we.abs()
    return y, m


def wgrad(G, x, dy, gather_x, gather_dy):
    dw = torch.zeros(G.N, x.shape[1], dy.shape[1], dtype=F64, device=x.device)
    m = torch.zeros_like(dw)
    for e, (p, n) in enumerate(zip(G.start, G.counts)):
        if n:
            a = (x[G.token(p, n)] if gather_x else x[p:p + n]).double()
            b = (dy[G.token(p, n)] if gather_dy else dy[p:p + n]).double()
            dw[e], m[e] = a.t() @ b, a.abs().t() @ b.abs()
    return dw, m


def sum_tol(n):
    """Error of an n-term fp32 sum of exact products on tensor cores, relative to the sum of magnitudes: a K = 16 step
    is off by at most 2^-20 (the router's certificate uses the same bound)."""
    return (n / 16 + 1) * 2.0 ** -20


def check(got, want, tol, what=""):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((got - want).abs().max()), got[bad][:4], want[bad][:4])
