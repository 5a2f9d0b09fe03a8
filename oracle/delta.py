"""Float64 oracles of the gated delta rule and of the join between blocks.

Plain NumPy from the definitions, one row at a time; no code is shared with the
GPU path.  Test infrastructure only.
"""

import numpy as np

UNIT_EPS = 1e-6


def _unit(x, unit):
    n = 1.0 / np.sqrt((x * x).sum(-1, keepdims=True) + UNIT_EPS) if unit else np.ones_like(x[..., :1])
    return x * n, n


def _lengths(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths]


def delta_forward(q, k, v, g, beta, h0=None, lengths=None, scale=None, unit=False):
    """``(y [B, T, Hv, Dv], hT [B, Hv, Dk, Dv])``, and the states after every row."""
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    scale = Dk ** -0.5 if scale is None else scale
    y = np.zeros((B, T, Hv, Dv))
    hT = np.zeros((B, Hv, Dk, Dv)) if h0 is None else h0.astype(np.float64).copy()
    for b, n in enumerate(_lengths(lengths, B, T)):
        for h in range(Hv):
            S = hT[b, h]
            for t in range(n):
                qt, _ = _unit(q[b, t, h // (Hv // Hk)].astype(np.float64), unit)
                kt, _ = _unit(k[b, t, h // (Hv // Hk)].astype(np.float64), unit)
                S = np.exp(float(g[b, t, h])) * S
                u = float(beta[b, t, h]) * (v[b, t, h].astype(np.float64) - S.T @ kt)
                S = S + np.outer(kt, u)
                y[b, t, h] = scale * (S.T @ qt)
            hT[b, h] = S
    return y, hT


def delta_backward(q, k, v, g, beta, dy, h0=None, lengths=None, dhT=None, scale=None, unit=False):
    """``(dq, dk, dv, dg, dbeta, dh0)`` by the chain rule through every row."""
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    scale = Dk ** -0.5 if scale is None else scale
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    dg, dbeta = np.zeros(g.shape), np.zeros(g.shape)
    dh0 = np.zeros((B, Hv, Dk, Dv)) if dhT is None else dhT.astype(np.float64).copy()
    for b, n in enumerate(_lengths(lengths, B, T)):
        for h in range(Hv):
            hk = h // (Hv // Hk)
            S = np.zeros((Dk, Dv)) if h0 is None else h0[b, h].astype(np.float64)
            seen = []
            for t in range(n):
                kt, _ = _unit(k[b, t, hk].astype(np.float64), unit)
                decayed = np.exp(float(g[b, t, h])) * S
                w = v[b, t, h].astype(np.float64) - decayed.T @ kt
                S = decayed + np.outer(kt, float(beta[b, t, h]) * w)
                seen.append((decayed, w, S))
            dS = dh0[b, h]
            for t in reversed(range(n)):
                decayed, w, S = seen[t]
                bt = float(beta[b, t, h])
                qt, nq = _unit(q[b, t, hk].astype(np.float64), unit)
                kt, nk = _unit(k[b, t, hk].astype(np.float64), unit)
                d = scale * dy[b, t, h].astype(np.float64)
                dqt = S @ d
                dS = dS + np.outer(qt, d)
                du = dS.T @ kt
                dbeta[b, t, h] = du @ w
                dw = bt * du
                dkt = dS @ (bt * w) - decayed @ dw
                dv[b, t, h] = dw
                dS = dS - np.outer(kt, dw)
                dg[b, t, h] = (dS * decayed).sum()
                dS = np.exp(float(g[b, t, h])) * dS
                if unit:
                    dqt, dkt = nq * (dqt - qt * (qt @ dqt)), nk * (dkt - kt * (kt @ dkt))
                dq[b, t, hk] += dqt
                dk[b, t, hk] += dkt
            dh0[b, h] = dS
    return dq, dk, dv, dg, dbeta, dh0


def _act(kind, g):
    with np.errstate(over="ignore"):
        s = np.where(g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))
    o = np.where(g >= 0, np.exp(-np.abs(g)), 1.0) / (1.0 + np.exp(-np.abs(g)))        # 1 - s
    return (s, s * o) if kind == "sigmoid" else (g * s, s + g * s * o)


def join_forward(h, r=None, gate=None, w_post=None, w_pre=None, post=True, pre=True, activation="silu", scale=1.0,
                 eps=1e-6):
    """``(y, x, n1, n2)``; x is None without ``pre``."""
    h = h.astype(np.float64)
    n1 = 1.0 / np.sqrt((h * h).mean(-1) + eps) if post else np.ones(len(h))
    p = h * n1[:, None] * (1.0 if w_post is None else w_post.astype(np.float64))
    if gate is not None:
        p = p * _act(activation, gate.astype(np.float64))[0]
    y = scale * p + (0.0 if r is None else r.astype(np.float64))
    if not pre:
        return y, None, n1, np.ones(len(h))
    n2 = 1.0 / np.sqrt((y * y).mean(-1) + eps)
    return y, y * n2[:, None] * (1.0 if w_pre is None else w_pre.astype(np.float64)), n1, n2


def join_backward(h, y, n1, n2, dy=None, dx=None, gate=None, w_post=None, w_pre=None, post=True, activation="silu",
                  scale=1.0):
    """``(dh, dr, dgate, dw_post, dw_pre)`` from the stored rows and factors."""
    h, y = h.astype(np.float64), y.astype(np.float64)
    n1, n2 = n1.astype(np.float64)[:, None], n2.astype(np.float64)[:, None]
    d = np.zeros_like(h) if dy is None else dy.astype(np.float64)
    dw_pre = None
    if dx is not None:
        z, c = y * n2, dx.astype(np.float64)
        dw_pre = (c * z).sum(0)
        c = c * (1.0 if w_pre is None else w_pre.astype(np.float64))
        d = d + n2 * (c - z * (c * z).mean(-1, keepdims=True))
    t, w = h * n1, 1.0 if w_post is None else w_post.astype(np.float64)
    e, dgate = scale * d, None
    if gate is not None:
        a, slope = _act(activation, gate.astype(np.float64))
        dgate = e * w * t * slope
        e = e * a
    dw_post = (e * t).sum(0)
    e = e * w
    dh = n1 * (e - t * (e * t).mean(-1, keepdims=True)) if post else e
    return dh, d, dgate, dw_post, dw_pre
