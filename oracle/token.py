"""Float64 oracles of the token-side operators: embedding, gated recurrence, distillation.

Plain NumPy from the definitions, one row or step at a time; no code is shared
with the GPU path.  Test infrastructure only.
"""

import numpy as np


def embed_forward(ids, table, scale):
    """``y[n] = scale * table[ids[n]]``; ids outside the table give zero rows."""
    V, D = table.shape
    y = np.zeros((len(ids), D))
    for n, v in enumerate(ids):
        if 0 <= v < V:
            y[n] = scale * table[v].astype(np.float64)
    return y


def embed_backward(ids, dy, V, scale):
    """``dE[v] = scale * sum of the dy rows of token v``."""
    dE = np.zeros((V, dy.shape[1]))
    for n, v in enumerate(ids):
        if 0 <= v < V:
            dE[v] += dy[n].astype(np.float64)
    return scale * dE


def sigmoid(v):
    with np.errstate(over="ignore"):
        e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def _lengths(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths]


def recur_forward(x, g, h0=None, lengths=None):
    """``h_t = sigmoid(g_t) h_{t-1} + sigmoid(-g_t) x_t``; ``(y, hT)``."""
    B, T, D = x.shape
    y = np.zeros((B, T, D))
    hT = np.zeros((B, D)) if h0 is None else h0.astype(np.float64).copy()
    for b, n in enumerate(_lengths(lengths, B, T)):
        for t in range(n):
            gt = g[b, t].astype(np.float64)
            hT[b] = sigmoid(gt) * hT[b] + sigmoid(-gt) * x[b, t].astype(np.float64)
            y[b, t] = hT[b]
    return y, hT


def recur_backward(x, g, dy, h0=None, lengths=None, dhT=None):
    """``(dx, dg, dh0)`` by the chain rule through ``h_t = f h_{t-1} + (1 - f) x_t``."""
    B, T, D = x.shape
    y, _ = recur_forward(x, g, h0, lengths)
    dx, dg = np.zeros((B, T, D)), np.zeros((B, T, D))
    dh = np.zeros((B, D)) if dhT is None else dhT.astype(np.float64).copy()
    for b, n in enumerate(_lengths(lengths, B, T)):
        for t in reversed(range(n)):
            gt = g[b, t].astype(np.float64)
            f, u = sigmoid(gt), sigmoid(-gt)
            before = y[b, t - 1] if t > 0 else (np.zeros(D) if h0 is None else h0[b].astype(np.float64))
            d = dh[b] + dy[b, t].astype(np.float64)
            dx[b, t] = u * d
            dg[b, t] = f * u * (before - x[b, t].astype(np.float64)) * d
            dh[b] = f * d
    return dx, dg, dh


def _row(z, ids, t, tau):
    """Student log-probabilities, lse, and the teacher's entries ``(id, log p)`` of a row."""
    V = len(z)
    z = z.astype(np.float64) / tau
    keep = [(int(i), float(v) / tau) for i, v in zip(ids, t) if 0 <= i < V and v != -np.inf]
    m = z.max()
    if not keep or m == -np.inf:
        return None, m, []
    log_s = np.log(np.exp(z - m).sum())       # beside z - m, not m: m may be the lowest float32
    tv = np.array([v for _, v in keep])
    tm = tv.max()
    lp = tv - (tm + np.log(np.exp(tv - tm).sum()))
    return z - m - log_s, m + log_s, list(zip([i for i, _ in keep], lp))


def distill(z, ids, t, tau, weight=None, dloss=None):
    """``(loss, lse, dz)``; a row of weight 0 has its ``lse`` all the same."""
    N, V = z.shape
    loss, lse, dz = np.zeros(N), np.zeros(N), np.zeros((N, V))
    for b in range(N):
        w = 1.0 if weight is None else float(weight[b])
        lq, lse[b], entries = _row(z[b], ids[b], t[b], tau)
        if w == 0.0 and lq is not None:
            continue
        if lq is None:
            if lse[b] != -np.inf:
                s = z[b].astype(np.float64) / tau
                lse[b] = s.max() + np.log(np.exp(s - s.max()).sum())
            continue
        q = np.exp(lq)
        for i, lp in entries:
            if np.exp(lp) > 0:
                loss[b] += np.exp(lp) * (lp - lq[i])
            q[i] -= np.exp(lp)
        loss[b] *= w * tau * tau
        dz[b] = q * w * tau * (1.0 if dloss is None else float(dloss[b]))
    return loss, lse, dz
