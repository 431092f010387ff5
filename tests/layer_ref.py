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
