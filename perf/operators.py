"""Workloads of the 4-bit expert path: residual + RMS norm, routing by scores,
microscaled (MX) 4-bit quantisation and the grouped expert FFN on 4-bit operands.

own = False computes each operator in elementary torch operations, in 32 bits,
rounded once at the end; own = True calls the library.

An MX e2m1 tensor is a pair (codes, scales): blocks of 32 along the last
dimension share a power of two 2^(scale - 127); codes hold two 4-bit values a
byte, the even element in the low half.  A block's exponent is
floor(log2(largest magnitude)) - 2; values round to the nearest of 0, 0.5, 1,
1.5, 2, 3, 4, 6 (ties to the even mantissa) and saturate at 6.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token through a large router (sigmoid scores, balance bias, 8 groups of 32, 4 kept): decode
        dict(name="route-sig-1", op="route", T=1, N=256, k=8, sigmoid=True, bias=True, groups=8, top_groups=4, top2=True,
             renorm=True),
        # a prefill batch of a softmax router without groups
        dict(name="route-soft-8192", op="route", T=8192, N=128, k=8, sigmoid=False, bias=False, groups=1, top_groups=1,
             top2=False, renorm=True),
        # the largest prefill batch of the grouped router
        dict(name="route-sig-131072", op="route", T=131072, N=256, k=8, sigmoid=True, bias=True, groups=8, top_groups=4,
             top2=True, renorm=True),
        # activations of a small odd batch, and of a long prefill, to 4 bits
        dict(name="quant-37", op="quant", rows=37, K=2048),
        dict(name="quant-16448", op="quant", rows=16448, K=7168),
        # bf16 expert weights [experts, K, features] to 4 bits along K, once per model load
        dict(name="quant-weights", op="quantw", N=128, K=2048, F=1536),
        # the norm before the layer: one token; a prefill batch with the 4-bit rows the experts take
        dict(name="norm-1", op="norm", T=1, H=4096, mx=False),
        dict(name="norm-mx-16448", op="norm", T=16448, H=7168, mx=True),
        # expert FFN: one token of the 8-expert layer (weight bytes), a decode batch and a prefill batch of the
        # 128-expert layer, a prefill batch of the 8-expert layer (operations)
        dict(name="ffn-mix-1", op="ffn", T=1, H=4096, N=8, k=2, I=14336, B=64),
        dict(name="ffn-qw-512", op="ffn", T=512, H=2048, N=128, k=8, I=768, B=16),
        dict(name="ffn-qw-8192", op="ffn", T=8192, H=2048, N=128, k=8, I=768, B=16),
        dict(name="ffn-mix-4096", op="ffn", T=4096, H=4096, N=8, k=2, I=14336, B=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        case = _draw(rng)
        if 3072 not in (*case.values(), 2 * case.get("I", 0)):   # no size of that kind in this repository
            return case


def _draw(rng):
    op = rng.choice(["route", "quant", "quantw", "norm", "ffn", "ffn"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        N = groups * rng.randint(2, 256 // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, top_groups * (N // groups)))
        return dict(op=op, T=_log(rng, 1, 131072), N=N, k=k, sigmoid=rng.random() < 0.6, bias=rng.random() < 0.5,
                    groups=groups, top_groups=top_groups, top2=rng.random() < 0.5, renorm=rng.random() < 0.7)
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 16448), K=32 * _log(rng, 1, 224))
    if op == "quantw":
        return dict(op=op, N=rng.randint(1, 64), K=32 * rng.randint(1, 64), F=8 * rng.randint(1, 192))
    if op == "norm":
        return dict(op=op, T=_log(rng, 1, 16448), H=32 * rng.randint(1, 224), mx=rng.random() < 0.5)
    H, I = 128 * rng.randint(1, 32), 128 * rng.randint(1, 32)
    N = _log(rng, 1, 128)
    while N > 1 and N * H * I > 400_000_000:
        N //= 2
    k = rng.randint(1, min(8, N))
    return dict(op=op, T=_log(rng, 1, 4096), H=H, N=N, k=k, I=I, B=rng.choice([8, 16, 32, 64, 128]))


def work(case):
    op = case["op"]
    if op == "route":
        T, N, k = case["T"], case["N"], case["k"]
        return {"bytes": 4 * T * N + 8 * T * k + 4 * N, "flops": 4 * T * N}
    if op == "quant":
        n = case["rows"] * case["K"]
        return {"bytes": 4 * n, "flops": 3 * n}
    if op == "quantw":
        n = case["N"] * case["K"] * case["F"]
        return {"bytes": 4 * n, "flops": 3 * n}
    if op == "norm":
        n = case["T"] * case["H"]
        return {"bytes": (10 if case["mx"] else 8) * n + 2 * case["H"], "flops": 7 * n}
    T, H, N, k, I = (case[x] for x in ("T", "H", "N", "k", "I"))
    mx = 0.5 + 1 / 32
    touched = N * (1 - (1 - k / N) ** T)
    return {"bytes": mx * 3 * H * I * touched + mx * T * H + 2 * T * k * H, "flops": 6 * T * k * H * I}


# ------------------------------------------------------------------ MX e2m1, plain form
def _mx_parts(x):
    """x fp32 [..., K]: signed grid values v (0 .. 6) and scale bytes per block of 32."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    byte = ((amax.view(torch.int32) >> 23) - 2).clamp(min=0)        # floor(log2 amax) - 2 + 127
    bad = ~torch.isfinite(amax)
    byte = torch.where(bad, 255, byte)
    inv = ((254 - byte.clamp(max=253)) << 23).view(torch.float32)   # 2^(127 - byte)
    v = b.abs() * inv
    m = 0.5 * ((v > 0.25).float() + (v >= 0.75).float() + (v > 1.25).float() + (v >= 1.75).float())
    m += (v > 2.5).float() + (v >= 3.5).float() + 2.0 * (v > 5.0).float()
    m = torch.where(bad, 0.0, m)
    return torch.where(torch.signbit(b) & ~bad, -m, m), byte


def _mx_values(x):
    """x rounded to MX e2m1, in fp32."""
    v, byte = _mx_parts(x)
    return (v * _pow2(byte)).reshape(x.shape)


def _pow2(byte):
    """2^(byte - 127) of integer scale bytes; 255 is NaN."""
    p = torch.where(byte == 0, 0x00400000, byte << 23).to(torch.int32).view(torch.float32)
    return torch.where(byte == 255, float("nan"), p)


def _mx_codes(x):
    v, byte = _mx_parts(x)
    a = v.abs()
    c = ((a >= 0.5).int() + (a >= 1).int() + (a >= 1.5).int() + (a >= 2).int() + (a >= 3).int() + (a >= 4).int()
         + (a >= 6).int() + 8 * torch.signbit(v).int()).reshape(*x.shape[:-1], -1, 2)
    return (c[..., 0] | (c[..., 1] << 4)).to(torch.uint8), byte.squeeze(-1).to(torch.uint8)


def _mx_expand(codes, scales):
    """(codes [..., K/2], scales [..., K/32]) -> fp32 [..., K]."""
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = lut[c.int()].reshape(*scales.shape, 32) * _pow2(scales.int()).unsqueeze(-1)
    return v.reshape(c.shape)


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


def _scores64(case, logits, bias):
    s = logits.double()
    s = torch.sigmoid(s) if case["sigmoid"] else torch.softmax(s, -1)
    return s, s if bias is None else s + bias.double()


def _margin(case, logits, bias):
    """Smallest relative distance to another choice of groups or experts, per token."""
    _, b = _scores64(case, logits, bias)
    G, N, k, tg = case["groups"], case["N"], case["k"], case["top_groups"]
    near = torch.full((b.shape[0],), math.inf, dtype=torch.float64, device=b.device)

    def gap(v, n):
        if n >= v.shape[-1]:
            return near
        t = v.topk(n + 1, -1).values
        return (t[:, n - 1] - t[:, n]) / t[:, n - 1].abs().clamp(min=1e-30)

    if G > 1:
        gb = b.reshape(-1, G, N // G)
        gs = gb.topk(2, -1).values.sum(-1) if case["top2"] else gb.amax(-1)
        near = torch.minimum(near, gap(gs, tg))
        kept = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, gs.topk(tg, -1).indices, True)
        b = torch.where(kept.unsqueeze(-1), gb, -math.inf).reshape(-1, N)
        if k == tg * (N // G):
            return near
    return torch.minimum(near, gap(b, k))


def _layout(idx, N, B):
    """Stable padded blocks of expert segments (moe_dispatch_align's layout)."""
    T, k = idx.shape
    R = T * k
    flat = idx.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=N)
    padded = (counts + B - 1) // B * B
    start, first = padded.cumsum(0) - padded, counts.cumsum(0) - counts
    e = flat[order]
    row = start[e] + torch.arange(R, device=DEV) - first[e]
    P = int(padded.sum())
    ids = torch.full((R + N * (B - 1),), R, dtype=torch.int32, device=DEV)
    ids[row] = order.int()
    blocks = torch.zeros(R // B + N, dtype=torch.int32, device=DEV)
    blocks[:P // B] = torch.repeat_interleave(torch.arange(N, device=DEV), padded // B).int()
    return dict(ids=ids, blocks=blocks, num_padded=torch.tensor([P], dtype=torch.int32, device=DEV), P=P,
                counts=counts, most=int(counts.max()))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case, op=op)
    if op == "route":
        T, N, k = case["T"], case["N"], case["k"]
        bias = 0.05 * _randn(g, N) * (1.0 if case["sigmoid"] else 0.02) if case["bias"] else None
        logits = _randn(g, T, N)
        # Tokens whose choice hangs on less than the resolution of 32-bit scores have no answer that every
        # correct evaluation shares: they are drawn again.
        for _ in range(20):
            near = (_margin(case, logits, bias) < 2e-5).nonzero().squeeze(-1)
            if near.numel() == 0:
                break
            logits[near] = _randn(g, near.numel(), N)
        s.update(logits=logits, bias=bias)
        if own:
            import invariant_expert_routing_gb300 as moe
            s["cfg"] = moe.make_config(128, N, k, 128, 8)
            s["scoring"] = moe.make_scoring(
                score=moe.MOE_SCORE_SIGMOID if case["sigmoid"] else moe.MOE_SCORE_SOFTMAX,
                num_groups=case["groups"], top_groups=case["top_groups"],
                group_score=moe.MOE_GROUP_TOP2_SUM if case["top2"] else moe.MOE_GROUP_MAX,
                renormalize=case["renorm"], scale=2.5)
            s["idx"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
            s["gate"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
    elif op in ("quant", "quantw"):
        if op == "quant":
            rows, K = case["rows"], case["K"]
            s["x"] = _hidden(g, rows, K)
        else:
            rows, K = case["N"] * case["F"], case["K"]
            s["x"] = torch.empty(case["N"], K, case["F"], dtype=torch.bfloat16, device=DEV)
            for e in range(case["N"]):
                s["x"][e] = 0.02 * _randn(g, K, case["F"])
        if own:
            lead = (rows,) if op == "quant" else (case["N"], case["F"])
            s["codes"] = torch.empty((*lead, K // 2), dtype=torch.uint8, device=DEV)
            s["scales"] = torch.empty((*lead, K // 32), dtype=torch.uint8, device=DEV)
            s["values"] = torch.empty((*lead, K), dtype=torch.bfloat16, device=DEV)
    elif op == "norm":
        T, H = case["T"], case["H"]
        s.update(x=_hidden(g, T, H), r=_hidden(g, T, H), w=(1.0 + 0.2 * _randn(g, H)).bfloat16())
        if own:
            for n in ("r_out", "out") + (("values",) if case["mx"] else ()):
                s[n] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
            s["codes"] = torch.empty((T, H // 2), dtype=torch.uint8, device=DEV) if case["mx"] else None
            s["scales"] = torch.empty((T, H // 32), dtype=torch.uint8, device=DEV) if case["mx"] else None
    else:
        T, H, N, k, I, B = (case[x] for x in ("T", "H", "N", "k", "I", "B"))
        s["x"], s["xs"] = _mx_codes(_hidden(g, T, H).float())
        s["w13"] = torch.empty(N, 2 * I, H // 2, dtype=torch.uint8, device=DEV)
        s["w13s"] = torch.empty(N, 2 * I, H // 32, dtype=torch.uint8, device=DEV)
        s["w2"] = torch.empty(N, H, I // 2, dtype=torch.uint8, device=DEV)
        s["w2s"] = torch.empty(N, H, I // 32, dtype=torch.uint8, device=DEV)
        for e in range(N):
            s["w13"][e], s["w13s"][e] = _mx_codes(0.02 * _randn(g, 2 * I, H))
            s["w2"][e], s["w2s"][e] = _mx_codes(0.02 * _randn(g, H, I))
        pull = 0.5 * _randn(g, N) - torch.log(-torch.log(torch.rand(T, N, generator=g, device=DEV).clamp(1e-6, 1 - 1e-6)))
        idx = pull.topk(k, -1).indices.sort(-1).values.int()
        s.update(_layout(idx, N, B))
        if own:
            import invariant_expert_routing_gb300 as moe
            s["cfg"] = moe.make_config(H, N, k, I, B)
            s["y"] = torch.zeros((s["ids"].numel(), H), dtype=torch.bfloat16, device=DEV)
            s["ws"] = moe.workspace_mx(s["cfg"], T, DEV)
            # the weights' scales are laid out once, where the weights are loaded
            s["w13p"], s["w2p"] = torch.empty_like(s["w13s"]), torch.empty_like(s["w2s"])
            moe.moe_pack_scales_mx(s["w13s"], s["w13p"], gate_up=True)
            moe.moe_pack_scales_mx(s["w2s"], s["w2p"], gate_up=False)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import invariant_expert_routing_gb300 as moe
    op = s["op"]
    if op == "route":
        moe.moe_route_scored(s["cfg"], s["scoring"], s["logits"], s["bias"], s["idx"], s["gate"])
        return {"idx": s["idx"], "gate": s["gate"]}
    if op == "quant":
        moe.moe_quantize_mx(s["x"], s["codes"], s["scales"])
        moe.moe_dequantize_mx(s["codes"], s["scales"], s["values"])
        return s["values"]
    if op == "quantw":
        moe.moe_quantize_weights_mx(s["x"], s["codes"], s["scales"])
        moe.moe_dequantize_mx(s["codes"], s["scales"], s["values"])
        return s["values"]
    if op == "norm":
        moe.moe_add_norm(s["x"], s["r"], s["w"], EPS, s["r_out"], s["out"], s["codes"], s["scales"])
        if not s["case"]["mx"]:
            return {"residual": s["r_out"], "out": s["out"]}
        moe.moe_dequantize_mx(s["codes"], s["scales"], s["values"])
        return {"residual": s["r_out"], "out": s["out"], "values": s["values"]}
    moe.moe_expert_ffn_mx(s["cfg"], s["x"], s["xs"], s["w13"], s["w13p"], s["w2"], s["w2p"], None, None, None, None,
                          s["ids"], s["blocks"], s["num_padded"], s["y"], None, s["ws"])
    return s["y"]   # rows without a route stay as they were: zeros


def _run_plain(s):
    case, op = s["case"], s["op"]
    if op == "route":
        N, k, G, tg = (case[x] for x in ("N", "k", "groups", "top_groups"))
        l = s["logits"]
        if case["sigmoid"]:
            score = 1.0 / (1.0 + torch.exp(-l))
        else:
            ex = torch.exp(l - l.amax(-1, keepdim=True))
            score = ex / ex.sum(-1, keepdim=True)
        b = score if s["bias"] is None else score + s["bias"]
        if G > 1:
            gb = b.reshape(-1, G, N // G)
            gs = gb.topk(2, -1).values.sum(-1) if case["top2"] else gb.amax(-1)
            kept = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, gs.topk(tg, -1).indices, True)
            b = torch.where(kept.unsqueeze(-1), gb, -math.inf).reshape(-1, N)
        idx = b.topk(k, -1).indices.sort(-1).values
        gate = score.gather(1, idx)
        if case["renorm"]:
            gate = gate / (gate.sum(-1, keepdim=True) + 1e-20)
        return {"idx": idx.int(), "gate": 2.5 * gate}
    if op == "quant":
        return _mx_values(s["x"].float()).bfloat16()
    if op == "quantw":
        return _mx_values(s["x"].transpose(1, 2).float().contiguous()).bfloat16()
    if op == "norm":
        v = s["x"].float() + s["r"].float()
        n = (v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * s["w"].float()).bfloat16()
        if not case["mx"]:
            return {"residual": v.bfloat16(), "out": n}
        return {"residual": v.bfloat16(), "out": n, "values": _mx_values(n.float()).bfloat16()}
    # expert FFN: every touched expert's rows in one batched product
    I, k, B, P = case["I"], case["k"], case["B"], s["P"]
    ids = s["ids"][:P].long()
    valid = ids < case["T"] * k
    touched = (s["counts"] > 0).nonzero().squeeze(-1)
    of = torch.repeat_interleave(s["blocks"][:P // B].long(), B)
    padded = (s["counts"] + B - 1) // B * B
    place = torch.arange(P, device=DEV) - (padded.cumsum(0) - padded)[of]
    at = (torch.searchsorted(touched, of) * s["most"] + place)[valid]
    x = _mx_expand(s["x"], s["xs"])
    rows = torch.zeros(touched.numel() * s["most"], x.shape[1], device=DEV)
    rows[at] = x[ids[valid] // k]
    gu = torch.bmm(rows.reshape(touched.numel(), s["most"], -1),
                   _mx_expand(s["w13"][touched], s["w13s"][touched]).transpose(1, 2))
    gate, up = gu[..., :I], gu[..., I:]
    a = _mx_values((gate / (1.0 + torch.exp(-gate)) * up).contiguous())
    y = torch.bmm(a, _mx_expand(s["w2"][touched], s["w2s"][touched]).transpose(1, 2))
    out = torch.zeros(s["ids"].numel(), x.shape[1], dtype=torch.bfloat16, device=DEV)
    out[:P][valid] = y.reshape(-1, y.shape[-1])[at].bfloat16()
    return out


# ------------------------------------------------------------------ the definitions, in 64 bits
def _round64(x):
    """x fp64 [..., K] rounded to MX e2m1 by the spacing of the grid around each value."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    e = torch.frexp(b.abs().amax(-1, keepdim=True)).exponent - 1       # floor(log2 amax)
    unit = torch.ldexp(torch.ones_like(b[..., :1]), (e - 2).clamp(min=-127))
    v = b / unit
    step = torch.ldexp(torch.ones_like(v), (torch.frexp(v.abs()).exponent - 1).clamp(min=0) - 1)
    q = (torch.round(v / step) * step).clamp(-6, 6)
    return (q * unit).reshape(x.shape)


def _expand64(codes, scales):
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=codes.device)
    out = torch.empty(*codes.shape, 2, dtype=torch.float64, device=codes.device)
    for half, c in ((0, codes & 15), (1, codes >> 4)):
        out[..., half] = torch.where(c >= 8, -1.0, 1.0).double() * grid[(c & 7).long()]
    v = out.reshape(*scales.shape, 32)
    return torch.ldexp(v, scales.int().unsqueeze(-1) - 127).reshape(*codes.shape[:-1], -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        N, k, G, tg = (case[x] for x in ("N", "k", "groups", "top_groups"))
        score, b = _scores64(case, s["logits"], s["bias"])
        if G > 1:
            best = b.reshape(-1, G, N // G).sort(-1, descending=True).values
            gs = best[..., 0] + best[..., 1] if case["top2"] else best[..., 0]
            rank = gs.argsort(dim=-1, descending=True, stable=True).argsort(-1)
            b = b.masked_fill((rank >= tg).repeat_interleave(N // G, 1), -math.inf)
        idx = b.argsort(dim=-1, descending=True, stable=True)[:, :k].sort(-1).values
        gate = score.gather(1, idx)
        if case["renorm"]:
            gate = gate / gate.sum(-1, keepdim=True)
        return {"idx": idx.int(), "gate": 2.5 * gate}
    if op == "quant":
        return _round64(s["x"].double())
    if op == "quantw":
        return torch.stack([_round64(w.double().t().contiguous()) for w in s["x"]])
    if op == "norm":
        v = s["x"].double() + s["r"].double()
        n = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * s["w"].double()
        if not case["mx"]:
            return {"residual": v, "out": n}
        return {"residual": v, "out": n, "values": _round64(n.bfloat16().double())}
    I, k = case["I"], case["k"]
    x = _expand64(s["x"], s["xs"])
    y = torch.zeros(s["ids"].numel(), case["H"], dtype=torch.float64, device=DEV)
    row = 0
    for e, n in enumerate(s["counts"].tolist()):
        if n:
            gu = x[s["ids"][row:row + n].long() // k] @ _expand64(s["w13"][e], s["w13s"][e]).t()
            a = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
            y[row:row + n] = _round64(a) @ _expand64(s["w2"][e], s["w2s"][e]).t()
        row += (n + case["B"] - 1) // case["B"] * case["B"]
    return y
