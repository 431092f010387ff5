"""The token-row operators in 64 bits on torch tensors, and the bounds that their tests hold the library to.

Bounds (u = half a step of the element type, relative): a product's fp32 sum of K terms is off by at most K 2^-23 times the
sum of the terms' magnitudes (an addition that truncates loses one unit in the last place of a partial sum, which no
ordering lets exceed that sum); fp32 operands as three bf16 planes leave out less than 2^-24 of it (each plane holds 8 bits
and its rounding leaves at most 2^-9, 2^-18 and 2^-27 of the value: the products left out are mid lo, lo mid, lo lo and
those with the last remainder, at most 5 2^-27 together, and the five smaller passes add K terms of at most 2^-8 each).
"""

from __future__ import annotations

import math

import numpy as np
import torch

U = {torch.bfloat16: 2.0**-9 * 2, torch.float16: 2.0**-12 * 2, torch.float32: 2.0**-24}
# (torch.finfo(t).eps / 2: 2^-8, 2^-11, 2^-24)


def pieces(col8, row, seed, offset):
    """uint64 [len, 8]: the generator's 16-bit pieces for arrays of column groups and rows, in unsigned 64-bit arithmetic."""
    u = np.uint64
    m = u(0xFFFFFFFF)
    c = [np.asarray(col8, dtype=u), np.asarray(row, dtype=u)]
    c += [np.full(c[0].shape, offset & 0xFFFFFFFF, dtype=u), np.full(c[0].shape, offset >> 32, dtype=u)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> u(32)) ^ c[1] ^ u(k[0]), b & m, (a >> u(32)) ^ c[3] ^ u(k[1]), a & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack([h for w in c for h in (w & u(0xFFFF), w >> u(16))], -1)


def keep_mask(T, N, p, seed, offset):
    """bool [T, N]: the elements that dropout keeps."""
    G = (N + 7) // 8
    bits = pieces(np.tile(np.arange(G), T), np.repeat(np.arange(T), G), seed, offset).reshape(T, G * 8)[:, :N]
    return bits >= np.uint64(math.floor(p * 65536 + 0.5))


def keep_mask_at(col8, row, cut, seed, offset):
    return pieces([col8], [row], seed, offset)[0] >= np.uint64(cut)


def drop_factor(T, N, p, seed, offset, device):
    cut = math.floor(p * 65536 + 0.5)
    if cut == 0:
        return torch.ones((T, N), dtype=torch.float64, device=device)
    return torch.from_numpy(keep_mask(T, N, p, seed, offset).astype(np.float64)).to(device) * (65536.0 / (65536 - cut))


def act(z, kind):
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if kind == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, kind):
    if kind == "relu":
        return (z > 0).double()
    if kind == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def sum_bound(K, dtype):
    """Of a K-term product, relative to the sum of its terms' magnitudes."""
    return K * 2.0**-23 * (1 + 2.0**-5 if dtype == torch.float32 else 1) + (2.0**-24 if dtype == torch.float32 else 0)


ACT_ERR = 2.0**-18  # of |z|: the functions' few units of 2^-23 and the rounding of their arguments
LIPSCHITZ = 1.13    # no activation here is steeper


def linear(x, w, bias, residual, kind, p, seed, offset):
    """(y, pre, bound of y, bound of pre) in float64."""
    dt, (T, K), N = x.dtype, x.shape, w.shape[0]
    X, W = x.double(), w.double()
    z = X @ W.T
    mag = X.abs() @ W.abs().T
    if bias is not None:
        z = z + bias.double()
        mag = mag + bias.double().abs()
    dz = sum_bound(K + 1, dt) * mag
    f = drop_factor(T, N, p, seed, offset, x.device)
    y = act(z, kind) * f
    err = (LIPSCHITZ * dz + (ACT_ERR * z.abs() if kind in ("gelu", "silu") else 0)) * f + 2.0**-22 * y.abs()
    if residual is not None:
        y = y + residual.double()
        err = err + 2.0**-23 * (residual.double().abs() + y.abs())
    tiny = 2.0**-25 if dt == torch.float16 else 0.0  # half a step of fp16's smallest numbers
    return y, z, err * (1 + U[dt]) + U[dt] * y.abs() + tiny, dz * (1 + U[dt]) + U[dt] * z.abs() + tiny


def linear_backward(x, w, dy, pre, kind, p, seed, offset):
    """(dx, dw, db), (their bounds) in float64."""
    dt, (T, K), N = x.dtype, x.shape, w.shape[0]
    X, W = x.double(), w.double()
    d = dy.double() * drop_factor(T, N, p, seed, offset, x.device)
    tiny = 2.0**-25 if dt == torch.float16 else 0.0
    err = 2.0**-22 * d.abs()
    if kind != "none":
        z = pre.double()
        err = err * LIPSCHITZ + (8 * ACT_ERR * (1 + z.abs()) if kind in ("gelu", "silu") else 0) * d.abs()
        d = d * act_slope(z, kind)
    round_d = err + (U[dt] if dt != torch.float32 else 0) * d.abs() + tiny  # dz as an operand of the products
    dx, dw, db = d @ W, d.T @ X, d.sum(0)
    ex = round_d @ W.abs() + sum_bound(N, dt) * ((d.abs() + round_d) @ W.abs())
    ew = round_d.T @ X.abs() + sum_bound(T, dt) * ((d.abs() + round_d).T @ X.abs())
    eb = err.sum(0) + T * 2.0**-23 * d.abs().sum(0)
    fin = lambda v, e: e * (1 + U[dt]) + U[dt] * v.abs() + tiny  # noqa: E731
    return (dx, dw, db), (fin(dx, ex), fin(dw, ew), fin(db, eb))


def logits(x, w, bias):
    z = x.double() @ w.double().T
    mag = x.double().abs() @ w.double().abs().T
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    return z, sum_bound(x.shape[1] + 1, x.dtype) * mag


def cross_entropy(x, w, labels, bias):
    """(loss, lse), bound (of either) in float64; rows without a label zero."""
    T, V = x.shape[0], w.shape[0]
    z, dz = logits(x, w, bias)
    has = labels >= 0
    lse = torch.logsumexp(z, 1) * has
    picked = z.gather(1, labels.clamp(min=0)[:, None])[:, 0]
    loss = (lse - picked) * has
    # each exponential off by its argument's error (|z| 2^-22 for the change of base, 2^-21 for the function), the sum of
    # them by the additions of 32 values, of at most V / 32 partial sums and of the join
    err = dz.max(1).values * 2 + (z.abs().max(1).values + 1) * 2.0**-21 + (64 + V / 32) * 2.0**-23 + 2.0**-22 * lse.abs()
    return (loss, lse), err * has


def cross_entropy_backward(x, w, labels, lse, dloss, bias):
    """(dx, dw, db), (their bounds) in float64."""
    dt, (T, D), V = x.dtype, x.shape, w.shape[0]
    z, dz = logits(x, w, bias)
    has = (labels >= 0)[:, None]
    q = torch.exp(z - lse.double()[:, None])
    rel = dz + (z.abs() + lse.double().abs()[:, None] + 2) * 2.0**-21
    e = q * rel
    q = q.clone()
    q[torch.arange(T, device=x.device), labels.clamp(min=0)] -= 1.0
    g = dloss.double()[:, None]
    q, e = torch.where(has, q * g, 0.0), torch.where(has, e * g.abs() + 2.0**-23 * (q * g).abs(), 0.0)
    if dt != torch.float32:
        e = e + U[dt] * (q.abs() + e)
    if dt == torch.float16:
        # dz is scaled by a power of two that brings the largest |dloss| to at least 2^14: half a step of the smallest fp16
        e = e + has * 2.0**-25 * dloss[labels >= 0].abs().max().double() * 2.0**-14 if has.any() else e
    X, W = x.double(), w.double()
    dx, dw, db = q @ W, q.T @ X, q.sum(0)
    ex = e @ W.abs() + 2 * sum_bound(V, dt) * ((q.abs() + e) @ W.abs())
    ew = e.T @ X.abs() + sum_bound(T, dt) * ((q.abs() + e).T @ X.abs())
    eb = e.sum(0) + T * 2.0**-23 * q.abs().sum(0)
    tiny = 2.0**-25 if dt == torch.float16 else 0.0
    fin = lambda v, b: b * (1 + U[dt]) + U[dt] * v.abs() + tiny  # noqa: E731
    return (dx, dw, db), (fin(dx, ex), fin(dw, ew), fin(db, eb))


def worst(got, want, bound):
    """The largest |got - want| in units of its bound (0 / 0 counts as 0)."""
    d = (got.double() - want).abs()
    r = torch.where(d == 0, 0.0, d / bound.clamp(min=1e-300))
    assert not torch.isnan(r).any(), "NaN where the definition has none"
    return float(r.max()) if r.numel() else 0.0
