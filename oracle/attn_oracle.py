"""fp64 numpy restatement of the packed attention and of the head norm with
rotary positions, straight from the formulas in include/flce.h."""
from __future__ import annotations

import numpy as np


def _sequences(cu, tokens):
    """The [lo, hi) of the sequences; none when the offsets do not ascend in [0, tokens]."""
    cu = [int(c) for c in cu]
    if any(c < 0 or c > tokens for c in cu) or any(b < a for a, b in zip(cu, cu[1:])):
        return []
    return [(a, b) for a, b in zip(cu, cu[1:]) if b > a]


def _probabilities(q, k, lo, hi, scale):
    s = scale * (q[lo:hi] @ k[lo:hi].T)
    s[np.triu_indices(hi - lo, 1)] = -np.inf
    m = s.max(axis=1, keepdims=True)
    e = np.exp(s - m)
    l = e.sum(axis=1, keepdims=True)
    return e / l, (m + np.log(l))[:, 0]


def attention_forward(q, k, v, cu, scale):
    """out [T, Hq, D], lse [Hq, T]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    T, HQ, _ = q.shape
    group = HQ // k.shape[1]
    out, lse = np.zeros_like(q), np.full((HQ, T), -np.inf)
    for lo, hi in _sequences(cu, T):
        for h in range(HQ):
            p, lse[h, lo:hi] = _probabilities(q[:, h], k[:, h // group], lo, hi, scale)
            out[lo:hi, h] = p @ v[lo:hi, h // group]
    return out, lse


def attention_backward(dout, q, k, v, cu, scale):
    """(dq, dk, dv) of sum(dout * out)."""
    dout, q, k, v = (np.asarray(x, np.float64) for x in (dout, q, k, v))
    T, HQ, _ = q.shape
    group = HQ // k.shape[1]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for lo, hi in _sequences(cu, T):
        for h in range(HQ):
            g = h // group
            p, _ = _probabilities(q[:, h], k[:, g], lo, hi, scale)
            do = dout[lo:hi, h]
            dv[lo:hi, g] += p.T @ do
            dp = do @ v[lo:hi, g].T
            ds = p * (dp - (p * dp).sum(axis=1, keepdims=True))
            dq[lo:hi, h] = scale * (ds @ k[lo:hi, g])
            dk[lo:hi, g] += scale * (ds.T @ q[lo:hi, h])
    return dq, dk, dv


def _pairs(rot, interleaved):
    j = np.arange(rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] turned by the angles cos, sin [T, rot / 2]."""
    y = x.copy()
    a, b = _pairs(2 * cos.shape[1], interleaved)
    c, s = cos[:, None, :], sin[:, None, :]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def qk_norm_rope_forward(x, w, cos, sin, positions, eps, interleaved=False):
    """One of q, k: R(position) (w * x / sqrt(mean(x^2) + eps))."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return _rotate(n * w, np.asarray(cos, np.float64)[positions],
                   np.asarray(sin, np.float64)[positions], interleaved)


def qk_norm_rope_backward(dy, x, w, cos, sin, positions, eps, interleaved=False):
    """(dx, dw) of sum(dy * y)."""
    dy, x, w = (np.asarray(t, np.float64) for t in (dy, x, w))
    g = _rotate(dy, np.asarray(cos, np.float64)[positions],
                -np.asarray(sin, np.float64)[positions], interleaved)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    gw = g * w
    return r * (gw - n * (gw * n).mean(-1, keepdims=True)), (g * n).sum(axis=(0, 1))
