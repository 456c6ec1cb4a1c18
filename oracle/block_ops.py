"""64-bit definitions of the operators between the recurrence and a training step, in numpy: the norm
of queries and keys with the position rotation, the gated feed-forward block, and the clipped policy
loss; forward and gradients.  The ``*_bounds`` functions give the magnitudes that the
rounding errors of an fp32 evaluation scale with.
"""
from __future__ import annotations

import numpy as np

from .layer_ops import sigmoid, silu, silu_grad


# ------------------------------------------------------------ norm and rotation
def _turn(x, pos, freq, inter, sign=1.0, bound=False):
    """Turns the first 2 len(freq) dimensions of x [T, H, d]; bound: |a| + |b| in both places."""
    if freq is None or len(freq) == 0:
        return np.abs(x) if bound else x.copy()
    R = 2 * len(freq)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if inter else (slice(0, R // 2), slice(R // 2, R))
    y = np.abs(x) if bound else x.copy()
    if bound:
        y[..., a] = y[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
        return y
    angle = pos.astype(np.float64)[:, None, None] * freq
    c, s = np.cos(angle), sign * np.sin(angle)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _unit(x, l2, eps):
    n = 1 if l2 else x.shape[-1]
    return 1 / np.sqrt((x * x).sum(-1, keepdims=True) / n + eps), n


def head_norm(x, w=None, pos=None, freq=None, inter=False, l2=False, eps=1e-6, bound=False):
    """One of q and k: x [T, H, d]."""
    r, _ = _unit(x, l2, eps)
    return _turn(x * r * (1 if w is None else w), pos, freq, inter, bound=bound)


def head_norm_backward(x, dy, w=None, pos=None, freq=None, inter=False, l2=False, eps=1e-6, bound=False):
    """dx, dw (dw also without a weight: that of ones)."""
    m = np.abs if bound else (lambda v: v)
    r, n = _unit(x, l2, eps)
    g = _turn(dy, pos, freq, inter, -1.0, bound)
    u = m(x * r)
    h = g * (1 if w is None else m(w))
    s = (h * u).sum(-1, keepdims=True) / n
    return r * (h + u * s if bound else h - u * s), (g * u).sum((0, 1))


# ------------------------------------------------------------ gated feed-forward block
def gelu(v):
    return v * sigmoid(np.sqrt(8 / np.pi) * (v + 0.044715 * v ** 3))


def gelu_grad(v):
    e = sigmoid(np.sqrt(8 / np.pi) * (v + 0.044715 * v ** 3))
    return e + v * e * (1 - e) * np.sqrt(8 / np.pi) * (1 + 3 * 0.044715 * v * v)


ACT = {"silu": (silu, silu_grad), "gelu": (gelu, gelu_grad)}


def glu(x, wg, wu, act="silu"):
    return ACT[act][0](x @ wg.T) * (x @ wu.T)


def glu_backward(x, wg, wu, dh, act="silu"):
    """dx, dwg, dwu."""
    f, df = ACT[act]
    g, u = x @ wg.T, x @ wu.T
    dg, du = dh * u * df(g), dh * f(g)
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x


# ------------------------------------------------------------ policy loss
def policy(z, y, old=None, adv=None, ref=None, lo=0.2, hi=0.2, kl=0.0, tau=1.0):
    """loss, lp, dloss/dlp and softmax of rows [R, V]; rows with y outside [0, V) are zero."""
    R, V = z.shape
    on = (y >= 0) & (y < V)
    t = z / tau
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = t.max(1, keepdims=True)
        e = np.exp(t - top)
        s = e.sum(1, keepdims=True)
        lp = (t - top)[np.arange(R), np.where(on, y, 0)] - np.log(s[:, 0])
        p = e / s
        if old is None:
            return None, np.where(on, lp, 0), None, p
        ratio = np.exp(lp - old)
        free, held = -adv * ratio, -adv * np.clip(ratio, 1 - lo, 1 + hi)
        loss, d = np.where(free < held, held, free), np.where(free < held, 0, free)
        loss, d = np.where(adv == 0, 0, loss), np.where(adv == 0, 0, d)
        if ref is not None:
            g = ref - lp
            loss, d = loss + kl * (np.exp(g) - g - 1), d + kl * (1 - np.exp(g))
    return np.where(on, loss, 0), np.where(on, lp, 0), np.where(on, d, 0), p


def policy_backward(z, y, dloss, **kw):
    """dlogits [R, V]."""
    _, _, d, p = policy(z, y, **kw)
    on = (y >= 0) & (y < z.shape[1])
    dz = np.where(on[:, None], -p, 0)
    dz[np.arange(len(y))[on], y[on]] += 1
    return np.where(on[:, None], dz * (d * dloss / kw.get("tau", 1.0))[:, None], 0)
