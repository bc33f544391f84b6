"""Workloads of the layer's training step: products grouped by expert with the gradients of their
inputs and weights, SwiGLU with gates and its gradient, and the norms before the layer with theirs.

own = False computes each operator in elementary torch operations, in 32 bits, rounded once at the
end; own = True calls the library.

Rows are grouped by expert as moe_dispatch_align lays them out: expert e's segment starts at the sum
of the earlier experts' row counts, each rounded up to a multiple of B, and holds counts[e] rows in
ascending route id r = t * k + j.  Rows that hold no route belong to nobody: they are not read
(prepare fills them with NaN) and not written.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the first expert product (gate and up columns) of a small batch, token rows fetched by route: latency
        dict(name="gemm-tiny-64", op="gemm", T=64, N=8, k=2, B=8, K=128, F=512, gather=True, transposed=False),
        # the same product of a long batch of the 128-expert layer
        dict(name="gemm-qw-8192", op="gemm", T=8192, N=128, k=8, B=16, K=2048, F=1536, gather=True, transposed=False),
        # gradient of the second product's input in the 8-expert layer: dy . W2^T, dy fetched by route
        dict(name="gemm-mix-4096-dx", op="gemm", T=4096, N=8, k=2, B=64, K=4096, F=14336, gather=True, transposed=True),
        # weight gradients: a short batch of odd sizes with bf16 gradients; the first product of the 128-expert layer
        # added to fp32 gradients of earlier batches; the second product of the 8-expert layer in bf16
        dict(name="wgrad-odd-333", op="wgrad", T=333, N=19, k=3, B=8, K=328, F=1000, gather_x=False, gather_dy=False,
             fp32=False, add=False),
        dict(name="wgrad-qw-8192-add", op="wgrad", T=8192, N=128, k=8, B=16, K=2048, F=1536, gather_x=True,
             gather_dy=False, fp32=True, add=True),
        dict(name="wgrad-mix-4096", op="wgrad", T=4096, N=8, k=2, B=64, K=14336, F=4096, gather_x=False,
             gather_dy=True, fp32=False, add=False),
        # the activation between the products: a serving batch of the 128-expert layer; its gradient in a long batch
        # of the 8-expert layer, the activation computed again beside it
        dict(name="swiglu-qw-512", op="swiglu", T=512, N=128, k=8, B=16, I=768, backward=False),
        dict(name="swiglu-mix-4096-backward", op="swiglu", T=4096, N=8, k=2, B=64, I=14336, backward=True),
        # residual + layer norm of one token and of a long prefill batch
        dict(name="norm-1", op="norm", T=1, H=4096),
        dict(name="norm-16448", op="norm", T=16448, H=7168),
        # gradients of the norms: an odd batch of the RMS norm, the longest batch of the layer norm
        dict(name="norm-37-backward", op="norm_backward", T=37, H=2048, centre=False),
        dict(name="norm-16448-backward", op="norm_backward", T=16448, H=7168, centre=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "wgrad", "wgrad", "swiglu", "norm", "norm_backward"])
    if op in ("norm", "norm_backward"):
        case = dict(op=op, T=_log(rng, 1, 16448), H=8 * _log(rng, 1, 896))
        if op == "norm_backward":
            case["centre"] = rng.random() < 0.5
        return case
    N = _log(rng, 1, 128)
    k = rng.randint(1, min(8, N))
    case = dict(op=op, T=_log(rng, 1, 8192), N=N, k=k, B=rng.choice([8, 16, 32, 64, 128]))
    if op == "swiglu":
        case.update(I=128 * _log(rng, 1, 64), backward=rng.random() < 0.6)
        return case
    case.update(K=8 * _log(rng, 2, 512), F=8 * _log(rng, 2, 512))
    while N * case["K"] * case["F"] > 400_000_000 or 2 * case["T"] * k * case["K"] * case["F"] > 9e11:
        case["K" if case["K"] > case["F"] else "F"] //= 16
        case["K"], case["F"] = 8 * max(2, case["K"] // 8), 8 * max(2, case["F"] // 8)
    if op == "gemm":
        case.update(gather=rng.random() < 0.5, transposed=rng.random() < 0.5)
    else:
        fp32 = rng.random() < 0.6
        gathered = rng.randint(0, 2)   # none, the input rows or the output gradient's rows
        case.update(gather_x=gathered == 1, gather_dy=gathered == 2, fp32=fp32, add=fp32 and rng.random() < 0.6)
    return case


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["T"] * case["H"]
        return {"bytes": 8 * n + 4 * case["H"], "flops": 9 * n}
    if op == "norm_backward":
        n = case["T"] * case["H"]
        return {"bytes": 8 * n + 10 * case["H"], "flops": 16 * n}
    T, N, k = case["T"], case["N"], case["k"]
    R = T * k
    if op == "swiglu":
        n = R * case["I"]
        return {"bytes": (12 if case["backward"] else 6) * n + 8 * R, "flops": (16 if case["backward"] else 6) * n}
    K, F = case["K"], case["F"]
    if op == "gemm":
        touched = N * (1 - (1 - k / N) ** T)
        return {"bytes": 2 * touched * K * F + 2 * (T if case["gather"] else R) * K + 2 * R * F, "flops": 2 * R * K * F}
    entry = (4 if case["fp32"] else 2) + (4 if case["add"] else 0)
    return {"bytes": entry * N * K * F + 2 * (T if case["gather_x"] else R) * K + 2 * (T if case["gather_dy"] else R) * F,
            "flops": 2 * R * K * F}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed & 0x7FFFFFFF)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _hidden(g, T, H):
    """Hidden states: unit normals with a few channels ten times larger, as trained models have."""
    ch = 1.0 + 9.0 * (torch.rand(H, generator=g, device=DEV) < 0.005).float()
    return _randn(g, T, H).mul_(ch).bfloat16()


def _layout(g, T, N, k, B):
    """Routes of a router whose experts differ in load, in moe_dispatch_align's layout."""
    pull = 0.5 * _randn(g, N) - torch.log(-torch.log(torch.rand(T, N, generator=g, device=DEV).clamp(1e-6, 1 - 1e-6)))
    flat = pull.topk(k, -1).indices.sort(-1).values.reshape(-1)
    R = T * k
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=N)
    padded = (counts + B - 1) // B * B
    start, first = padded.cumsum(0) - padded, counts.cumsum(0) - counts
    e = flat[order]
    row = start[e] + torch.arange(R, device=DEV) - first[e]
    ids = torch.full((R + N * (B - 1),), R, dtype=torch.int32, device=DEV)
    ids[row] = order.int()
    return dict(ids=ids, counts=counts.int(), num_padded=padded.sum().int().reshape(1), row=row, route=order, of=e,
                place=torch.arange(R, device=DEV) - first[e], rows=ids.numel(), segments=counts.tolist(),
                most=int(counts.max()))


def _rows(g, s, F, gathered, T):
    """Token rows [T, F], or grouped rows with NaN where there is no route."""
    if gathered:
        return _hidden(g, T, F)
    x = torch.full((s["rows"], F), float("nan"), dtype=torch.bfloat16, device=DEV)
    x[s["row"]] = _randn(g, s["row"].numel(), F).bfloat16()
    return x


def prepare(case, seed):
    g = _gen(seed)
    op, T = case["op"], case["T"]
    s = dict(case=case, op=op)
    if op in ("norm", "norm_backward"):
        H = case["H"]
        s.update(x=_hidden(g, T, H), r=_hidden(g, T, H), w=(1.0 + 0.2 * _randn(g, H)).bfloat16(),
                 b=(0.1 * _randn(g, H)).bfloat16())
        if op == "norm_backward":
            s["dy"] = _randn(g, T, H).bfloat16()
        if own:
            import invariant_expert_routing_gb300 as moe
            s["out"], s["dx"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
            if op == "norm_backward":
                s["dw"], s["db"] = torch.empty(H, device=DEV), torch.empty(H, device=DEV)
                s["ws"] = moe.workspace_norm_backward(T, H, DEV)
        return s
    N, k, B = case["N"], case["k"], case["B"]
    s.update(_layout(g, T, N, k, B))
    cfg = None
    if own:
        import invariant_expert_routing_gb300 as moe
        cfg = s["cfg"] = moe.make_config(128, N, k, case.get("I", 128), B)
        s["ws"] = moe.workspace_grouped(cfg, T, DEV)
    if op == "swiglu":
        I = case["I"]
        s["gu"] = _rows(g, s, 2 * I, False, T)
        gate = torch.rand(T, k, generator=g, device=DEV) + 0.05
        s["gate"] = gate / gate.sum(-1, keepdim=True)
        if case["backward"]:
            s["da"] = _rows(g, s, I, False, T)
        if own:
            s["a"] = torch.zeros((s["rows"], I), dtype=torch.bfloat16, device=DEV)
            if case["backward"]:
                s["dgu"] = torch.zeros((s["rows"], 2 * I), dtype=torch.bfloat16, device=DEV)
                s["dgate"] = torch.zeros((T, k), device=DEV)
    elif op == "gemm":
        K, F = case["K"], case["F"]
        s["x"] = _rows(g, s, K, case["gather"], T)
        s["w"] = torch.empty((N, F, K) if case["transposed"] else (N, K, F), dtype=torch.bfloat16, device=DEV)
        for e in range(N):
            s["w"][e] = 0.02 * _randn(g, *s["w"].shape[1:])
        if own:
            s["y"] = torch.zeros((s["rows"], F), dtype=torch.bfloat16, device=DEV)
    else:
        K, F = case["K"], case["F"]
        s["x"] = _rows(g, s, K, case["gather_x"], T)
        s["dy"] = _rows(g, s, F, case["gather_dy"], T)
        s["add"] = None
        if case["add"]:
            s["add"] = torch.empty((N, K, F), device=DEV)
            for e in range(N):
                s["add"][e] = 10.0 * _randn(g, K, F)
        if own:
            s["dw"] = torch.empty((N, K, F), dtype=torch.float32 if case["fp32"] else torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import invariant_expert_routing_gb300 as moe
    case, op = s["case"], s["op"]
    if op == "norm":
        moe.moe_add_layer_norm(s["x"], s["r"], s["w"], s["b"], EPS, s["dx"], s["out"])
        return {"residual": s["dx"], "out": s["out"]}
    if op == "norm_backward":
        # r: the gradient that reaches the residual past the norm
        db = s["db"] if case["centre"] else None
        moe.moe_norm_backward(s["x"], s["dy"], s["r"], s["w"], EPS, s["dx"], s["dw"], db, s["ws"],
                              centre=case["centre"])
        return {"dx": s["dx"], "dw": s["dw"], **({"db": db} if case["centre"] else {})}
    T = case["T"]
    if op == "swiglu":
        if not case["backward"]:
            moe.moe_swiglu(s["cfg"], T, s["gu"], s["gate"], s["ids"], s["num_padded"], s["a"])
            return s["a"]
        moe.moe_swiglu_backward(s["cfg"], T, s["gu"], s["gate"], s["da"], s["ids"], s["num_padded"], s["dgu"],
                                s["dgate"], s["a"])
        return {"dgu": s["dgu"], "dgate": s["dgate"], "a": s["a"]}
    if op == "gemm":
        moe.moe_grouped_gemm(s["cfg"], T, s["x"], s["w"], s["ids"], s["counts"], s["y"], s["ws"],
                             gather=case["gather"], transposed=case["transposed"])
        return s["y"]
    moe.moe_grouped_wgrad(s["cfg"], T, s["x"], s["dy"], s["ids"], s["counts"], s["dw"], s["ws"], dw_add=s["add"],
                          gather_x=case["gather_x"], gather_dy=case["gather_dy"])
    return s["dw"]


def _grouped(s, x, gathered):
    """The rows of every touched expert in one padded batch [experts, most, columns], fp32."""
    touched = torch.tensor([e for e, n in enumerate(s["segments"]) if n], device=DEV)
    at = torch.searchsorted(touched, s["of"]) * s["most"] + s["place"]
    rows = torch.zeros(touched.numel() * s["most"], x.shape[1], device=DEV)
    rows[at] = (x[s["route"] // s["case"]["k"]] if gathered else x[s["row"]]).float()
    return touched, at, rows.reshape(touched.numel(), s["most"], -1)


def _run_plain(s):
    case, op = s["case"], s["op"]
    if op == "norm":
        v = s["x"].float() + s["r"].float()
        d = v - v.mean(-1, keepdim=True)
        n = d / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS) * s["w"].float() + s["b"].float()
        return {"residual": v.bfloat16(), "out": n.bfloat16()}
    if op == "norm_backward":
        v, dy = s["x"].float(), s["dy"].float()
        if case["centre"]:
            v = v - v.mean(-1, keepdim=True)
        inv = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
        n = v * inv
        g = dy * s["w"].float()
        d = g - n * (g * n).mean(-1, keepdim=True)
        if case["centre"]:
            d = d - g.mean(-1, keepdim=True)
        out = {"dx": (s["r"].float() + d * inv).bfloat16(), "dw": (dy * n).sum(0)}
        return {**out, "db": dy.sum(0)} if case["centre"] else out
    if op == "swiglu":
        I, row = case["I"], s["row"]
        g, u = s["gu"][row, :I].float(), s["gu"][row, I:].float()
        w = s["gate"].reshape(-1)[s["route"]].unsqueeze(-1)
        sig = 1.0 / (1.0 + torch.exp(-g))
        a = torch.zeros((s["rows"], I), dtype=torch.bfloat16, device=DEV)
        a[row] = (w * (g * sig) * u).bfloat16()
        if not case["backward"]:
            return a
        da = s["da"][row].float()
        dgu = torch.zeros((s["rows"], 2 * I), dtype=torch.bfloat16, device=DEV)
        dgu[row] = torch.cat([w * da * u * sig * (1.0 + g * (1.0 - sig)), w * da * g * sig], -1).bfloat16()
        dgate = torch.zeros(case["T"] * case["k"], device=DEV)
        dgate[s["route"]] = (da * (g * sig) * u).sum(-1)
        return {"dgu": dgu, "dgate": dgate.reshape(case["T"], case["k"]), "a": a}
    if op == "gemm":
        touched, at, x = _grouped(s, s["x"], case["gather"])
        w = s["w"][touched].float()
        y = torch.bmm(x, w.transpose(1, 2) if case["transposed"] else w)
        out = torch.zeros((s["rows"], case["F"]), dtype=torch.bfloat16, device=DEV)
        out[s["row"]] = y.reshape(-1, case["F"])[at].bfloat16()
        return out
    touched, _, x = _grouped(s, s["x"], case["gather_x"])
    _, _, dy = _grouped(s, s["dy"], case["gather_dy"])
    dw = torch.zeros((case["N"], case["K"], case["F"]), device=DEV)
    dw[touched] = torch.bmm(x.transpose(1, 2), dy)
    if s["add"] is not None:
        dw = dw + s["add"]
    return dw if case["fp32"] else dw.bfloat16()


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        v = s["x"].double() + s["r"].double()
        std = torch.sqrt(v.var(-1, correction=0, keepdim=True) + EPS)
        return {"residual": v, "out": (v - v.mean(-1, keepdim=True)) / std * s["w"].double() + s["b"].double()}
    if op == "norm_backward":
        v, dy, w = s["x"].double(), s["dy"].double(), s["w"].double()
        H = case["H"]
        if case["centre"]:
            std = torch.sqrt(v.var(-1, correction=0, keepdim=True) + EPS)
            n = (v - v.mean(-1, keepdim=True)) / std
        else:
            std = torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)
            n = v / std
        g = dy * w
        inner = torch.einsum("th,th->t", g, n).unsqueeze(-1) / H
        d = (g - (g.mean(-1, keepdim=True) if case["centre"] else 0.0) - n * inner) / std
        out = {"dx": s["r"].double() + d, "dw": torch.einsum("th,th->h", dy, n)}
        return {**out, "db": dy.sum(0)} if case["centre"] else out
    starts, at = [], 0
    for n in s["segments"]:
        starts.append(at)
        at += (n + case["B"] - 1) // case["B"] * case["B"]
    if op == "swiglu":
        I = case["I"]
        a = torch.zeros((s["rows"], I), dtype=torch.float64, device=DEV)
        dgu = torch.zeros((s["rows"], 2 * I), dtype=torch.float64, device=DEV)
        dgate = torch.zeros(case["T"] * case["k"], dtype=torch.float64, device=DEV)
        for p, n in zip(starts, s["segments"]):
            g, u = s["gu"][p:p + n].double().split(I, -1)
            r = s["ids"][p:p + n].long()
            w = s["gate"].reshape(-1)[r].double().unsqueeze(-1)
            silu = g * torch.sigmoid(g)
            a[p:p + n] = w * silu * u
            if case["backward"]:
                da = s["da"][p:p + n].double()
                slope = torch.sigmoid(g) + silu * torch.sigmoid(-g)
                dgu[p:p + n] = w * torch.cat([da * u * slope, da * silu], -1)
                dgate[r] = torch.einsum("ri,ri->r", da, silu * u)
        return {"dgu": dgu, "dgate": dgate.reshape(case["T"], -1), "a": a} if case["backward"] else a

    def segment(x, gathered, p, n):
        return (x[s["ids"][p:p + n].long() // case["k"]] if gathered else x[p:p + n]).double()
    if op == "gemm":
        y = torch.zeros((s["rows"], case["F"]), dtype=torch.float64, device=DEV)
        for e, (p, n) in enumerate(zip(starts, s["segments"])):
            w = s["w"][e].double()
            y[p:p + n] = segment(s["x"], case["gather"], p, n) @ (w.t() if case["transposed"] else w)
        return y
    dw = torch.zeros((case["N"], case["K"], case["F"]), dtype=torch.float64, device=DEV)
    for e, (p, n) in enumerate(zip(starts, s["segments"])):
        dw[e] = segment(s["x"], case["gather_x"], p, n).t() @ segment(s["dy"], case["gather_dy"], p, n)
    return dw if s["add"] is None else dw.add_(s["add"])
