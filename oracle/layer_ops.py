"""64-bit definitions of the layer operators, forward and gradients, in numpy.

Each is the formula written out per sequence and token.  ``bound=True`` computes
instead the sum of the magnitudes of every term (inputs by absolute value, no
cancellation): the scale of an fp32 evaluation's rounding error, which the
tests multiply by a count of roundings.  For the scan's bound the decay rates
are halved: a product of decays exp(-r) with a relative error of r k units is off by
r exp(-r) k <= exp(-r / 2) k units, so the bound covers errors of the exponents.
"""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def silu(v):
    return v * sigmoid(v)


def silu_grad(v, bound=False):
    s = sigmoid(v)
    return s * (1 + (np.abs(v) if bound else v) * (1 - s))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def _seqs(cu):
    return [(n, int(cu[n]), int(cu[n + 1])) for n in range(len(cu) - 1)]


# ------------------------------------------------------------------ convolution
def conv(x, w, cu, b=None, state=None, act=True, bound=False):
    """y [T, D], state_out [N, W-1, D], pre-activations [T, D]."""
    T, D = x.shape
    W = w.shape[1]
    m = np.abs if bound else (lambda a: a)
    pre = np.zeros((T, D))
    tails = np.zeros((len(cu) - 1, W - 1, D))
    for n, lo, hi in _seqs(cu):
        full = np.concatenate([np.zeros((W - 1, D)) if state is None else state[n], x[lo:hi]])
        for t in range(hi - lo):
            for i in range(W):
                pre[lo + t] += m(w[:, i] * full[t + i])
        tails[n] = full[len(full) - (W - 1):]
    if b is not None:
        pre += m(b)
    return (silu(pre) if act and not bound else pre), tails, pre


def conv_backward(x, w, dy, cu, b=None, state=None, act=True, dstate_out=None, bound=False):
    """dx, dw, db, dstate_in."""
    T, D = x.shape
    W = w.shape[1]
    m = np.abs if bound else (lambda a: a)
    pre = conv(x, w, cu, b, state, act)[2]
    # the derivative is at most 1.1 and its own derivative at most 1: an error of pre enters by its own scale
    g = m(dy) * (silu_grad(pre, bound) if act else 1.0)
    if bound and act:
        g = g + np.abs(dy) * conv(x, w, cu, b, state, act, True)[2]
    dx, dw, db = np.zeros((T, D)), np.zeros((D, W)), np.zeros(D)
    ds = np.zeros((len(cu) - 1, W - 1, D))
    for n, lo, hi in _seqs(cu):
        L = hi - lo
        full = np.concatenate([np.zeros((W - 1, D)) if state is None else state[n], x[lo:hi]])
        dfull = np.zeros((L + W - 1, D))
        for t in range(L):
            for i in range(W):
                dfull[t + i] += m(w[:, i]) * g[lo + t]
                dw[:, i] += g[lo + t] * m(full[t + i])
            db += g[lo + t]
        if dstate_out is not None:
            dfull[L:] += m(dstate_out[n])
        ds[n], dx[lo:hi] = dfull[:W - 1], dfull[W - 1:]
    return dx, dw, db, ds


# ------------------------------------------------------------------------- scan
def _ssm_in(p, bound):
    m = np.abs if bound else (lambda a: a)
    v = p["dt"] + (p["dt_bias"] if p.get("dt_bias") is not None else 0.0)
    delta = softplus(v) if p.get("dt_softplus", True) else v
    A = -np.abs(p["A"]) / 2 if bound else p["A"]
    return m, v, m(delta), A


def _spread(g, D):
    """[G, S] -> [D, S]"""
    return np.repeat(g, D // g.shape[0], axis=0)


def ssm(p, cu, bound=False):
    """p: dict of x, dt, A, B, C and optionally D, z, dt_bias, dt_softplus, state_in.
    Returns y, state_out and the states after every token [T, D, S]."""
    m, _, delta, A = _ssm_in(p, bound)
    T, D = p["x"].shape
    S = A.shape[1]
    y, hs = np.zeros((T, D)), np.zeros((T, D, S))
    last = np.zeros((len(cu) - 1, D, S))
    for n, lo, hi in _seqs(cu):
        h = np.zeros((D, S)) if p.get("state_in") is None else m(p["state_in"][n])
        for t in range(lo, hi):
            h = np.exp(delta[t][:, None] * A) * h + (delta[t] * m(p["x"][t]))[:, None] * _spread(m(p["B"][t]), D)
            hs[t] = h
            y[t] = (h * _spread(m(p["C"][t]), D)).sum(1)
        last[n] = h
    if p.get("D") is not None:
        y = y + m(p["D"] * p["x"])
    if p.get("z") is not None:
        y = y * m(silu(p["z"]))
    return y, last, hs


def ssm_backward(p, dy, cu, dstate_out=None, bound=False):
    """Dict of dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dstate_in."""
    m, v, delta, A = _ssm_in(p, bound)
    T, D = p["x"].shape
    G, S = p["B"].shape[1:]
    _, _, hs = ssm(p, cu, bound)
    x, dy = m(p["x"]), m(dy)
    skip = m(p["D"]) if p.get("D") is not None else np.zeros(D)
    r = dict(dx=np.zeros((T, D)), ddt=np.zeros((T, D)), dA=np.zeros((D, S)), dB=np.zeros((T, G, S)),
             dC=np.zeros((T, G, S)), dD=np.zeros(D), dz=np.zeros((T, D)), ddt_bias=np.zeros(D),
             dstate_in=np.zeros((len(cu) - 1, D, S)))
    for n, lo, hi in _seqs(cu):
        e = np.zeros((D, S)) if dstate_out is None else m(dstate_out[n]).copy()
        for t in range(hi - 1, lo - 1, -1):
            Bt, Ct = _spread(m(p["B"][t]), D), _spread(m(p["C"][t]), D)
            d = dy[t]
            if p.get("z") is not None:
                raw = (hs[t] * Ct).sum(1) + skip * x[t]
                r["dz"][t] = dy[t] * raw * silu_grad(p["z"][t], bound)
                d = dy[t] * m(silu(p["z"][t]))
            g = Ct * d[:, None] + e
            before = hs[t - 1] if t > lo else (np.zeros((D, S)) if p.get("state_in") is None else m(p["state_in"][n]))
            a = np.exp(delta[t][:, None] * A)
            q = a * before
            r["dC"][t] = (hs[t] * d[:, None]).reshape(G, D // G, S).sum(1)
            r["dB"][t] = (g * (delta[t] * x[t])[:, None]).reshape(G, D // G, S).sum(1)
            gB = (g * Bt).sum(1)
            r["dx"][t] = delta[t] * gB + skip * d
            r["dD"] += d * x[t]
            r["dA"] += g * q * delta[t][:, None]
            dd = (g * q * (np.abs(p["A"]) if bound else A)).sum(1) + x[t] * gB
            r["ddt"][t] = dd * (sigmoid(v[t]) if p.get("dt_softplus", True) else 1.0)
            e = a * g
        r["dstate_in"][n] = e
    r["ddt_bias"] = r["ddt"].sum(0)
    return r


# ------------------------------------------------------------------- layer norm
def layer_norm(x, w, b=None, eps=1e-5):
    mean = x.mean(1)
    rstd = 1 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * w
    return (y if b is None else y + b), mean, rstd


def layer_norm_backward(x, w, dy, eps=1e-5):
    _, mean, rstd = layer_norm(x, w, None, eps)
    n = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - n * (g * n).mean(1, keepdims=True))
    return dx, (dy * n).sum(0), dy.sum(0)


def layer_norm_bounds(x, w, dy=None, eps=1e-5):
    """Magnitude sums of y, dx, dw, db, counting that an error of the mean, on the scale of mean |x|,
    enters n = (x - mean) rstd."""
    _, mean, rstd = layer_norm(x, w, None, eps)
    size = np.abs(x).mean(1, keepdims=True) * rstd[:, None]
    n = np.abs((x - mean[:, None]) * rstd[:, None]) + size
    y = n * np.abs(w)
    if dy is None:
        return y
    g = np.abs(dy * w)
    dx = rstd[:, None] * (g + g.mean(1, keepdims=True) + n * (g * n).mean(1, keepdims=True))
    return y, dx, (np.abs(dy) * n).sum(0), np.abs(dy).sum(0)
