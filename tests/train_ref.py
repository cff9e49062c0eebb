"""Plain 64-bit implementations (numpy) of the training operators declared in
include/dynconv_train.h, written from their formulas, and the bounds on what the
fp32 kernels may differ by, counted in half steps of fp32 (E = 2^-24 relative
per rounding)."""
from __future__ import annotations

import numpy as np

E = 2.0 ** -24


# ------------------------------------------------------------------- balance


def top_k(row, k):
    """Indices of the k largest, the lower index first among equals, NaN last."""
    key = np.where(np.isnan(row), -np.inf, row)
    order = sorted(range(len(row)), key=lambda i: (np.isnan(row[i]), -key[i], i))
    return order[:k]


def balance(alpha, mask, k, sigmoid, coef):
    """alpha [rows][groups][n] float64 -> dict(counts, mean, kept, loss)."""
    rows, groups, n = alpha.shape
    keep = np.ones(rows, bool) if mask is None else mask.astype(bool)
    a = alpha[keep]
    counts = np.zeros((groups, n), np.int64)
    for row in a:
        for j in range(groups):
            counts[j, top_k(row[j], k)] += 1
    M = a.shape[0]
    p = a
    if sigmoid:
        S = a.sum(-1, keepdims=True)
        p = np.divide(a, S, out=np.zeros_like(a), where=S != 0)
    mean = p.sum(0) / M if M else np.zeros((groups, n))
    loss = coef * n / (k * groups) * (counts / max(M, 1) * mean).sum()
    return dict(counts=counts, mean=mean, kept=M, loss=loss)


def balance_loss(alpha, mask, counts, k, sigmoid, coef):
    """The loss with the counts held fixed (what the gradient differentiates)."""
    rows, groups, n = alpha.shape
    a = alpha[np.ones(rows, bool) if mask is None else mask.astype(bool)]
    p = a / a.sum(-1, keepdims=True) if sigmoid else a
    M = a.shape[0]
    return coef * n / (k * groups) * (counts / M * p.mean(0)).sum()


def balance_grad(alpha, mask, counts, k, sigmoid, coef, dloss):
    """(gradient, the size of the terms that its fp32 form adds up)."""
    rows, groups, n = alpha.shape
    keep = np.ones(rows, bool) if mask is None else mask.astype(bool)
    M = int(keep.sum())
    out = np.zeros(alpha.shape)
    size = np.zeros(alpha.shape)
    if M == 0:
        return out, size
    c = dloss * coef * n / (k * groups) * counts / M ** 2
    if not sigmoid:
        out[keep] = c
        size[keep] = np.abs(c)
        return out, size
    a = alpha[keep]
    S = a.sum(-1, keepdims=True)
    p = np.divide(a, S, out=np.zeros_like(a), where=S != 0)
    dot = (c * p).sum(-1, keepdims=True)
    inv = np.divide(1.0, S, out=np.zeros_like(S), where=S != 0)
    out[keep] = (c - dot) * inv
    size[keep] = (np.abs(c) + np.abs(dot)) * np.abs(inv)
    return out, size


# --------------------------------------------------------------------- AdamW


def _mix(x):
    x = np.asarray(x, np.uint64) & np.uint64(0xFFFFFFFF)
    lo = np.uint64(0xFFFFFFFF)
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x9E3779B9)) & lo
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0x6A09E667)) & lo
    return x ^ (x >> np.uint64(16))


def dither(seed, step, place, numel, start=0):
    """u in [0, 1): 16 bits for every element from `start` (below 2^33) on."""
    lo = np.uint64(0xFFFFFFFF)
    key = _mix(_mix(_mix(seed) ^ (np.uint64(step) & lo)) ^ np.uint64(place))
    e = np.arange(start, start + numel, dtype=np.uint64)
    h = _mix(key ^ (e >> np.uint64(1)))
    u = np.where(e & np.uint64(1), h >> np.uint64(16), h & np.uint64(0xFFFF))
    return u.astype(np.float64) / 65536.0


def to_e4m3(y, u):
    """|y| to a neighbour on the e4m3 grid (fixed spacing 2^-9 below 2^-6)."""
    y = np.maximum(y, 0.0)
    step = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    return np.minimum(np.floor(y / step + u) * step, 448.0)


def to_bf16_dithered(x, u):
    a = np.abs(x)
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -126))) - 7)
    return np.copysign(np.floor(a / step + u) * step, x)


def blocks(x, fill=0.0):
    pad = -len(x) % 256
    return np.concatenate([x, np.full(pad, fill)]).reshape(-1, 256)


def widen(code, scale):
    return code * np.repeat(scale, 256)[:len(code)]


def adamw(p, g, m, v, *, lr, beta1, beta2, eps, step, decay, scale=1.0):
    """One step in 64 bits: (p, m, v, bounds of the fp32 kernel's p, m, v). The
    bounds count roundings: a product of a rounded constant two, a sum one more."""
    g = g * scale
    gE = 1 if scale != 1.0 else 0
    m1, v1 = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    m_terms = np.abs(beta1 * m) + np.abs((1 - beta1) * g)
    em = (3 + gE) * E * m_terms + 1e-44
    ev = (5 + 2 * gE) * E * v1 + 1e-44
    root = np.sqrt(v1 / (1 - beta2 ** step))
    size = lr / (1 - beta1 ** step)
    update = size * m1 / (root + eps)
    p1 = p * (1 - lr * decay) - update
    # quotient: the error of m over the denominator, and the denominator's own
    # (half of v's, the root, its constant, the sum), the division (two units in
    # the last place = 4 E), the rate's and the product's rounding
    rel_v = np.divide(ev, v1, out=np.zeros_like(v1), where=v1 > 0)
    ep = size * em / (root + eps) + np.abs(update) * (rel_v / 2 + 12 * E)
    ep = ep + 3 * E * np.abs(p) + 2 * E * np.abs(p1) + 1e-44
    return p1, m1, v1, ep, em, ev
