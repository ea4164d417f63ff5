"""fp64 numpy restatement of the layer norm, the rotary positions and the linear
distillation, straight from the formulas in include/flce.h."""
from __future__ import annotations

import numpy as np


def f64(x):
    return np.asarray(x, np.float64)


# --------------------------------------------------------------------- layer norm
def layer_norm_forward(s, w, b, eps, rms=False):
    """(y, mean, rstd) of the rows of s; w, b may be None."""
    s = f64(s)
    mean = np.zeros(s.shape[0]) if rms else s.mean(-1)
    rstd = 1.0 / np.sqrt(((s - mean[:, None]) ** 2).mean(-1) + eps)
    y = (s - mean[:, None]) * rstd[:, None]
    if w is not None:
        y = y * f64(w)
    if b is not None:
        y = y + f64(b)
    return y, mean, rstd


def layer_norm_backward(dy, s, w, eps, ds=None, rms=False):
    """(dx, dw, db) of sum(dy * y) + sum(ds * s)."""
    dy, s = f64(dy), f64(s)
    _, mean, rstd = layer_norm_forward(s, None, None, eps, rms)
    n = (s - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * f64(w)
    dx = g - n * (g * n).mean(-1, keepdims=True)
    if not rms:
        dx = dx - g.mean(-1, keepdims=True)
    dx = dx * rstd[:, None]
    if ds is not None:
        dx = dx + f64(ds)
    return dx, (dy * n).sum(0), dy.sum(0)


# --------------------------------------------------------------------- rotary positions
def rope(x, inv_freq, positions, magnitude=1.0, interleaved=False, backward=False):
    """x [T, H, D] with its first 2 * len(inv_freq) values turned by positions * inv_freq."""
    x, inv_freq = f64(x), f64(inv_freq)
    angle = np.array([[float(int(p)) * f for f in inv_freq] for p in positions]).reshape(len(positions), -1)
    if backward:
        angle = -angle
    c, s = magnitude * np.cos(angle)[:, None], magnitude * np.sin(angle)[:, None]
    half = len(inv_freq)
    j = np.arange(half)
    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


# --------------------------------------------------------------------- distillation
def teacher(ids, t, temperature, V, teacher_lse=None):
    """(q [N, K], log q, valid [N]): the teacher's probabilities of the entries, 0 where
    there is none; a row with an id of V or more counts as one without entries."""
    ids, t = np.asarray(ids), f64(t) / temperature
    there = (ids >= 0) & ~(t == -np.inf)
    valid = there.any(-1) & ~(ids >= V).any(-1)
    there &= valid[:, None]
    t = np.where(there, t, -np.inf)
    if teacher_lse is None:
        # relative to the largest, before the sum's logarithm could be lost in it
        t = t - np.where(valid, t.max(-1, initial=-np.inf), 0.0)[:, None]
        with np.errstate(divide="ignore"):
            tl = np.log(np.exp(t).sum(-1))
        tl = np.where(valid, tl, 0.0)
    else:
        tl = f64(teacher_lse)
    logq = np.where(there, t - tl[:, None], -np.inf)
    return np.exp(logq), logq, valid


def distill_forward(X, W, ids, t, temperature=1.0, reduction="mean", teacher_lse=None):
    """(loss, row losses, lse, logits at the ids (0 where there is none), valid count)."""
    ids, V = np.asarray(ids), len(W)
    z = f64(X) @ f64(W).T
    q, logq, valid = teacher(ids, t, temperature, V, teacher_lse)
    m = (z / temperature).max(-1)
    lse = m + np.log(np.exp(z / temperature - m[:, None]).sum(-1))
    known = (ids >= 0) & (ids < V)
    logits = np.where(known, np.take_along_axis(z, np.where(known, ids, 0), 1), 0.0)
    logp = logits / temperature - lse[:, None]
    rows = np.where(q > 0, q * (np.where(q > 0, logq, 0.0) - logp), 0.0).sum(-1)
    n = int(valid.sum())
    loss = rows.sum() / (max(n, 1) if reduction == "mean" else 1)
    return loss, rows, lse, logits, n


def distill_backward(X, W, ids, t, temperature=1.0, reduction="mean", teacher_lse=None, grad_loss=1.0):
    """(dX, dW)."""
    X, W, ids = f64(X), f64(W), np.asarray(ids)
    _, _, lse, _, n = distill_forward(X, W, ids, t, temperature, reduction, teacher_lse)
    q, _, valid = teacher(ids, t, temperature, len(W), teacher_lse)
    dz = np.exp(X @ W.T / temperature - lse[:, None]) * q.sum(-1, keepdims=True)
    for i in range(len(X)):
        if valid[i]:
            for k in range(ids.shape[1]):
                if q[i, k] > 0:
                    dz[i, ids[i, k]] -= q[i, k]
    dz[~valid] = 0.0
    dz *= grad_loss / temperature / ((max(n, 1)) if reduction == "mean" else 1)
    return dz @ W, dz.T @ X
