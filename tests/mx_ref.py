"""The 4-bit expert path in 64 bits (numpy): microscaled e2m1 conversion,
residual + RMS norm, routing by scores and the expert FFN with an interval
around every value that fp32 arithmetic may round either way."""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _exponent(amax):
    """floor(log2(amax)) - 2, at least -127 (an all-zero block takes -127)."""
    _, e = np.frexp(amax)
    return np.where(amax > 0, np.maximum(e - 3, -127), -127)


def _to_grid(v):
    """|v| <= 8 to the nearest grid value, ties to the even mantissa, saturating at 6."""
    a = np.abs(v)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    return np.copysign(np.minimum(np.rint(a / step) * step, 6.0), v)   # rint: half to even


def quantize(x):
    """x [..., K] -> codes [..., K/2] uint8, scales [..., K/32] uint8."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    fin = np.where(bad[..., None], 0.0, b)
    e = _exponent(np.abs(fin).max(-1))
    q = _to_grid(np.ldexp(fin, -e[..., None]))
    code = np.searchsorted(GRID, np.abs(q)).astype(np.uint8) | (np.signbit(q).astype(np.uint8) << 3)
    code = np.where(bad[..., None], 0, code).astype(np.uint8).reshape(*x.shape[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), np.where(bad, 255, e + 127).astype(np.uint8)


def dequantize(codes, scales):
    codes, scales = np.asarray(codes), np.asarray(scales)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*scales.shape, 32)
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v * s[..., None]).reshape(*codes.shape[:-1], -1)


def norm(x, residual, weight, eps):
    v = x.astype(np.float64) + (0.0 if residual is None else residual.astype(np.float64))
    return v, v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)


def route(logits, bias, k, sigmoid, groups=1, top_groups=1, top2=False, renorm=False, scale=1.0):
    """(idx [T, k] ascending, gate [T, k], margin [T]): margin = smallest distance to another choice."""
    l = np.asarray(logits, np.float64)
    T, N = l.shape
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            m = np.fmax.reduce(l, axis=1, keepdims=True)
            m = np.where(np.isneginf(m), 0.0, m)
            ex = np.exp(l - m)
            tot = ex.sum(1, keepdims=True)
            s = ex / np.where(tot == 0, 1.0, tot)
    b = s if bias is None else s + np.asarray(bias, np.float64)
    idx, gate, margin = np.zeros((T, k), np.int32), np.zeros((T, k)), np.full(T, np.inf)

    def best(v, n):
        """Indices of the n best: larger first, equal by lower index, NaN last."""
        return sorted(range(len(v)), key=lambda i: (np.isnan(v[i]), -v[i] if not np.isnan(v[i]) else 0.0, i))[:n]

    for t in range(T):
        cand = np.arange(N)
        if groups > 1:
            size = N // groups
            gs = np.zeros(groups)
            for g in range(groups):
                v = b[t, g * size:(g + 1) * size]
                o = best(v, 2 if top2 else 1)
                gs[g] = v[o].sum()
            o = best(gs, groups)
            if top_groups < groups:
                margin[t] = min(margin[t], abs(gs[o[top_groups - 1]] - gs[o[top_groups]]))
            cand = np.concatenate([np.arange(g * size, (g + 1) * size) for g in sorted(o[:top_groups])])
        o = best(b[t, cand], len(cand))
        if k < len(cand):
            margin[t] = min(margin[t], abs(b[t, cand[o[k - 1]]] - b[t, cand[o[k]]]))
        idx[t] = np.sort(cand[o[:k]])
        gate[t] = s[t, idx[t]]
    if renorm:
        gate = gate / (gate.sum(1, keepdims=True) + 1e-20)
    return idx, scale * gate, margin


def _mx_interval(a, d):
    """Least and greatest value that each element of a, known to within +-d,
    may have after conversion: both neighbours of its own rounding and of its
    block's exponent."""
    shape = a.shape
    a, d = a.reshape(*shape[:-1], -1, 32), d.reshape(*shape[:-1], -1, 32)
    amax, dmax = np.abs(a).max(-1), d.max(-1)
    lo = np.full(a.shape, np.inf)
    hi = np.full(a.shape, -np.inf)
    for m in (np.maximum(amax - dmax, 0.0), amax + dmax):
        e = _exponent(m)[..., None]
        for v in (a - d, a + d):
            q = np.ldexp(_to_grid(np.clip(np.ldexp(v, -e), -8.0, 8.0)), e)
            lo, hi = np.minimum(lo, q), np.maximum(hi, q)
    return lo.reshape(shape), hi.reshape(shape)


def ffn_rows(x, w13, w2):
    """x [R, H], w13 [2I, H], w2 [H, I] (values of MX tensors) -> (y, tol):
    y in 64 bits and the bound of an fp32-accumulating evaluation.

    A sum of n products in fp32 blocks of 64 is off by at most (n/64 + 64)
    2^-23 of the sum of magnitudes (a tensor core may truncate); silu and the
    product add 2^-20 relative.  Where that interval holds a rounding boundary
    of the 4-bit conversion, the converted value is an interval too, and its
    width goes through W2.  The stored bf16 adds half a unit, 2^-8 relative."""
    H, I = x.shape[1], w2.shape[1]
    gu = x @ w13.T
    err = (H / 64 + 64) * 2.0 ** -23 * (np.abs(x) @ np.abs(w13).T)
    g, u, eg, eu = gu[:, :I], gu[:, I:], err[:, :I], err[:, I:]
    with np.errstate(over="ignore"):
        silu = g / (1.0 + np.exp(-g))
    a = silu * u
    d = 1.1 * eg * (np.abs(u) + eu) + (np.abs(silu) + 1.1 * eg) * eu + 2.0 ** -20 * np.abs(a)
    lo, hi = _mx_interval(a, d)
    q = dequantize(*quantize(a))
    y = q @ w2.T
    tol = (np.maximum(hi - q, q - lo)) @ np.abs(w2).T
    tol += (I / 64 + 64) * 2.0 ** -23 * (np.abs(q) @ np.abs(w2).T)
    return y, tol * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(y)
