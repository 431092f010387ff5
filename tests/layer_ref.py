"""The norm, the 8-bit projection, the gated feed-forward, the token log probabilities and distillation in 64 bits on torch
tensors, and the bounds that their tests hold the library to (rows_ref.py has the projection's and what they share).

Bounds, with u = half a step of the element type, relative:
  - a row's fp32 sum: a thread adds at most 64 values one after another and joins others' in at most 16 steps, each step
    rounding to half a unit (2^-24), the sum of magnitudes above it: 2^-17 of that sum covers it with its products;
  - 1 / sqrt: 2 units (2^-22), of an argument whose own error counts half;
  - the short exponential: 2^-21 of itself, and for an argument x the error of x log2(e), |x| 2^-22.
"""

from __future__ import annotations

import torch

import rows_ref as rows
from rows_ref import U

TINY = {torch.bfloat16: 0.0, torch.float16: 2.0**-25, torch.float32: 0.0}  # half a step of fp16's smallest numbers
E4M3 = 2.0**-4  # half a step of the 8-bit type, relative; its smallest numbers are 2^-9 apart


def worst(got, want, bound):
    """rows_ref.worst where infinities, or NaN, that agree count as 0."""
    got = got.double()
    same = (torch.isinf(want) & (got == want)) | (want.isnan() & got.isnan())
    return rows.worst(torch.where(same, 0.0, got), torch.where(same, 0.0, want), torch.where(same, 1.0, bound))


def rounded(v, err, dt):
    return err * (1 + U[dt]) + U[dt] * v.abs() + TINY[dt]


# ------------------------------------------------------------------------------------------ norm


def rms_norm(x, w, residual, eps):
    """(y, h), (their bounds), and the bound of y before it is rounded; in float64."""
    dt = x.dtype
    h = x.double() if residual is None else x.double() + residual.double()
    eh = 2.0**-24 * h.abs()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * w.double()
    ey = 2.0**-17 * y.abs()
    return (y, h), (rounded(y, ey, dt), rounded(h, eh, dt)), ey


def e4m3_bound(y, ey, scale):
    """Of q scale against y: a half step of what stands there, or of the smallest numbers."""
    return E4M3 * (y.abs() + ey) * (1 + 2.0**-16) + 2.0**-10 * (1 + 2.0**-16) * scale[:, None] + ey


def rms_norm_backward(h, w, dy, dh, eps):
    """(dx, dw), (their bounds) in float64."""
    dt, T = h.dtype, h.shape[0]
    H, W, Y = h.double(), w.double(), dy.double()
    f = 1 / torch.sqrt(H.square().mean(1, keepdim=True) + eps)
    n, g = H * f, Y * W
    dx = f * (g - n * (g * n).mean(1, keepdim=True))
    ex = 2.0**-16 * f * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
        ex = ex + 2.0**-23 * (dh.double().abs() + dx.abs())
    dw = (Y * n).sum(0)
    ew = (2.0**-17 + T * 2.0**-24) * (Y * n).abs().sum(0)
    return (dx, dw), (rounded(dx, ex, dt), rounded(dw, ew, dt))


# ------------------------------------------------------------------------------------------ log probabilities


def token_logprobs(z, labels, top):
    """(logp, lse, entropy, top_logp, top_idx) in float64 (and int64), (bounds of the first four)."""
    T, V = z.shape
    Z = z.double()
    m = Z.max(1).values
    bad = (Z.isnan() | torch.isposinf(Z)).any(1)  # rows without a value
    rest = torch.log(torch.exp(Z - m[:, None]).sum(1))  # apart from m, beside whose magnitude it may be nothing
    lse = torch.where(bad, float("nan"), m + rest)
    l = (Z - m[:, None]) - rest[:, None]
    d = (Z - m[:, None]).clamp(min=-1e30)
    p = torch.where(torch.isneginf(Z), 0.0, torch.exp(l))
    logp = l.gather(1, labels.clamp(min=0)[:, None])[:, 0]
    entropy = rest - (p * torch.where(p > 0, d, 0.0)).sum(1)
    far = (p * torch.where(p > 0, d.abs(), 0.0)).sum(1)
    far2 = (p * torch.where(p > 0, d.abs() * (1 + d.abs()), 0.0)).sum(1)
    es = 2.0**-20 + 2.0**-22 * far + (V / 256 + 64) * 2.0**-24  # of the sum of exponentials, relative
    rest = rest.abs()
    el = es + 2.0**-22 * (m.abs() + rest + 1)
    pick = lambda v: es.reshape(-1, *[1] * (v.dim() - 1)) + 2.0**-22 * (v.abs() + 2 * rest.reshape(-1, *[1] * (v.dim() - 1)) + 1)  # noqa: E731
    ee = es * (2 + far) + 2.0**-21 * far2 + (V / 256 + 64) * 2.0**-24 * far + 2.0**-22 * (rest + far + 1)
    order = Z + 0.0
    best, idx = torch.sort(order, dim=1, descending=True, stable=True)
    idx = idx[:, :top]
    top_logp = torch.where(bad[:, None], float("nan"), l.gather(1, idx))
    logp, entropy = torch.where(bad, float("nan"), logp), torch.where(bad, float("nan"), entropy)
    has = labels >= 0
    logp = torch.where(has, logp, 0.0)
    return (logp, lse, entropy, top_logp, idx), (pick(logp), el, ee, pick(top_logp))


def token_logprobs_backward(z, labels, lse, entropy, dlogp, dentropy):
    """dlogits and its bound in float64, for the lse and entropy that are given."""
    dt, V = z.dtype, z.shape[1]
    Z, L = z.double(), lse.double()[:, None]
    has = (labels >= 0) & (labels < V)
    g = torch.where(has, dlogp.double(), 0.0)[:, None]
    l = (Z - L).clamp(min=-1e4)
    p = torch.exp(l)
    c = g
    mag = g.abs()
    if dentropy is not None:
        h, H = dentropy.double()[:, None], entropy.double()[:, None]
        c = g + h * (l + H)
        mag = mag + h.abs() * (l.abs() + H.abs())
    d = -p * c
    one = torch.zeros_like(d).scatter_(1, labels.clamp(0, V - 1)[:, None], 1.0) * has[:, None]
    err = p * mag * (2.0**-19 + 2.0**-21 * (l.abs() + Z.abs().clamp(max=1e4) + L.abs().clamp(max=1e4))) + one * 2.0**-23 * (g.abs() + d.abs())
    d = d + one * g
    return d, rounded(d, err, dt)


# ------------------------------------------------------------------------------------------ the gated feed-forward


def gated_linear(x, w, bias, kind):
    """(y, pre), (their bounds) in float64. An activation is off by rows.ACT_ERR of its argument and no steeper than LIPSCHITZ."""
    dt, K, F = x.dtype, x.shape[1], w.shape[0] // 2
    z = x.double() @ w.double().T
    mag = x.double().abs() @ w.double().abs().T
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    ez = rows.sum_bound(K + 1, dt) * mag
    g, u, eg, eu = z[:, :F], z[:, F:], ez[:, :F], ez[:, F:]
    a = rows.act(g, kind)
    ea = rows.LIPSCHITZ * eg + (rows.ACT_ERR * g.abs() if kind in ("gelu", "silu") else 0)
    y = a * u
    ey = ea * (u.abs() + eu) + a.abs() * eu + 2.0**-22 * y.abs()
    return (y, z), (rounded(y, ey, dt), rounded(z, ez, dt))


def gated_linear_backward(x, w, dy, pre, kind):
    """(dx, dw, db), (their bounds) in float64; dz is an operand of the element type."""
    dt, T, F = x.dtype, x.shape[0], dy.shape[1]
    X, W, d = x.double(), w.double(), dy.double()
    g, u = pre.double()[:, :F], pre.double()[:, F:]
    a, s = rows.act(g, kind), rows.act_slope(g, kind)
    smooth = rows.ACT_ERR if kind in ("gelu", "silu") else 0.0
    dz = torch.cat([d * u * s, d * a], 1)
    err = torch.cat([(d * u).abs() * 8 * smooth * (1 + g.abs()), d.abs() * smooth * g.abs()], 1) + 2.0**-21 * dz.abs()
    once = err + (U[dt] if dt != torch.float32 else 0) * dz.abs() + TINY[dt]
    dx, dw, db = dz @ W, dz.T @ X, dz.sum(0)
    ex = once @ W.abs() + rows.sum_bound(2 * F, dt) * ((dz.abs() + once) @ W.abs())
    ew = once.T @ X.abs() + rows.sum_bound(T, dt) * ((dz.abs() + once).T @ X.abs())
    eb = err.sum(0) + T * 2.0**-23 * dz.abs().sum(0)
    return (dx, dw, db), (rounded(dx, ex, dt), rounded(dw, ew, dt), rounded(db, eb, dt))


# ------------------------------------------------------------------------------------------ 8-bit rows


def linear_q8(x, xs, w, ws, bias, residual, kind, dt):
    """y and its bound in float64: the products are exact, an fp32 sum of K of them is off by K 2^-23 of their magnitudes."""
    K = x.shape[1]
    X, W = x.float().double(), w.float().double()
    scale = torch.outer(xs.double(), ws.double())
    z, ez = (X @ W.T) * scale, (K * 2.0**-23 + 2.0**-22) * (X.abs() @ W.abs().T) * scale
    if bias is not None:
        z = z + bias.double()
        ez = ez + 2.0**-23 * (z.abs() + bias.double().abs())
    y = rows.act(z, kind)
    ey = rows.LIPSCHITZ * ez + (rows.ACT_ERR * z.abs() if kind in ("gelu", "silu") else 0)
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2.0**-23 * (residual.double().abs() + y.abs())
    return y, rounded(y, ey, dt)


# ------------------------------------------------------------------------------------------ distillation


def targets(idx, values, temperature, V):
    """(Q [T, V] float64: the teacher's probabilities, its entropy's terms q ln q summed, rows with a target)."""
    there = (idx >= 0) & ~torch.isneginf(values)
    v = torch.where(there, values.double() / temperature, float("-inf"))
    has = there.any(1)
    q = torch.where(has[:, None] & there, torch.softmax(torch.where(has[:, None], v, 0.0), 1), 0.0)
    Q = torch.zeros(idx.shape[0], V, dtype=torch.float64, device=idx.device).scatter_add_(1, idx.clamp(0, V - 1), q)
    return q, Q, has


def _share_error(idx, values, temperature):
    """Of a q, relative: the exponential's, its argument's and the division's."""
    there = (idx >= 0) & ~torch.isneginf(values)
    return 2.0**-20 + 2.0**-21 * torch.where(there, values.double().abs() / temperature, 0.0).amax(1)


def distill(x, w, idx, values, bias, temperature):
    """(loss, lse), (their bounds) in float64; rows without a target zero."""
    V = w.shape[0]
    z, dz = rows.logits(x, w, bias)
    z, dz = z / temperature, dz / temperature
    q, _, has = targets(idx, values, temperature, V)
    lse = torch.logsumexp(z, 1)
    logp = (z - lse[:, None]).gather(1, idx.clamp(0, V - 1))
    gap = torch.where(q > 0, torch.log(q.clamp(min=1e-300)) - logp, 0.0)
    loss = (q * gap).sum(1)
    el = dz.max(1).values * 2 + (z.abs().max(1).values + 1) * 2.0**-21 + (64 + V / 32) * 2.0**-23 + 2.0**-22 * lse.abs()
    far = (z.abs().max(1).values + lse.abs())
    eloss = el + dz.max(1).values + (q * (gap.abs() + 1)).sum(1) * (_share_error(idx, values, temperature) + 2.0**-20) + 2.0**-21 * far
    return (loss * has, lse * has), (eloss * has, el * has)


def distill_backward(x, w, idx, values, lse, dloss, bias, temperature):
    """(dx, dw, db), (their bounds) in float64, for the lse that is given."""
    dt, (T, D), V = x.dtype, x.shape, w.shape[0]
    z, dz = rows.logits(x, w, bias)
    z, dz = z / temperature, dz / temperature
    _, Q, has = targets(idx, values, temperature, V)
    p = torch.exp(z - lse.double()[:, None])
    g = (dloss.double() / temperature)[:, None]
    d = torch.where(has[:, None], (p - Q) * g, 0.0)
    e = p * (dz + (z.abs() + lse.double().abs()[:, None] + 2) * 2.0**-21) + Q * _share_error(idx, values, temperature)[:, None]
    # (an exponential below fp32's smallest normal number comes as 0: off by 2^-126 at most)
    e = torch.where(has[:, None], (e + 2.0**-126) * g.abs() + 2.0**-22 * (p + Q) * g.abs(), 0.0)
    free = e.clone()
    if dt != torch.float32:
        e = e + U[dt] * (d.abs() + e)
    if dt == torch.float16 and bool(has.any()):
        # dz is scaled by a power of two that brings the largest |dloss| / temperature to at least 2^14
        e = e + has[:, None] * 2.0**-25 * g[has].abs().max() * 2.0**-14
    X, W = x.double(), w.double()
    dx, dw, db = d @ W, d.T @ X, d.sum(0)
    ex = e @ W.abs() + 2 * rows.sum_bound(V, dt) * ((d.abs() + e) @ W.abs())
    ew = e.T @ X.abs() + rows.sum_bound(T, dt) * ((d.abs() + e).T @ X.abs())
    eb = free.sum(0) + T * 2.0**-23 * d.abs().sum(0)
    return (dx, dw, db), (rounded(dx, ex, dt), rounded(dw, ew, dt), rounded(db, eb, dt))
