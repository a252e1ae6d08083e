"""CPU fp64 references of what stands around the experts: layer norm and the router's gate, each with
its gradient written from the formula (tests check the formulas against differences)."""
from __future__ import annotations

import numpy as np


def layer_norm(x, gamma, beta, eps):
    """x [T, d] -> (y, mean [T], rstd [T], xhat)."""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    xhat = (x - mean[:, None]) * rstd[:, None]
    y = xhat * (1.0 if gamma is None else gamma) + (0.0 if beta is None else beta)
    return y, mean, rstd, xhat


def layer_norm_grad(dy, x, gamma, eps):
    """(dx, dgamma, dbeta) of sum(dy * y)."""
    dy = np.asarray(dy, np.float64)
    _, _, rstd, xhat = layer_norm(x, gamma, None, eps)
    g = dy * (1.0 if gamma is None else gamma)
    dx = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) - xhat * (g * xhat).mean(axis=1, keepdims=True))
    return dx, (dy * xhat).sum(axis=0), dy.sum(axis=0)


def gate(logits, mask, k, renorm):
    """The gate of [T, E] logits, token by token. Returns a dict: ids and weights [T, k], lse [T] (-inf:
    the token takes no part), p [T, E] (0 there), counts [E], n, prob_sum [E], loss [2]."""
    lg = np.asarray(logits, np.float64)
    T, E = lg.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    lse = np.full(T, -np.inf)
    p = np.zeros((T, E))
    for t in range(T):
        row = lg[t]
        if (mask is not None and not mask[t]) or np.all(row == -np.inf):
            continue
        with np.errstate(invalid="ignore"):
            top = row.max()  # NaN if there is one
            e = np.exp(row - top)
            s = e.sum()
            lse[t] = top + np.log(s)
            p[t] = e / s
        order = sorted((i for i in range(E) if row[i] > -np.inf), key=lambda i: (-row[i], i))[:k]
        ids[t, :len(order)] = order
        w[t, :len(order)] = p[t, order]
        if renorm:
            w[t] /= w[t].sum()
    on = lse != -np.inf
    n = int(on.sum())
    counts = np.bincount(ids[ids >= 0], minlength=E)
    prob = p.sum(axis=0)
    loss = np.zeros(2)
    if n:
        loss[0] = E * ((counts / (k * n)) * (prob / n)).sum()
        loss[1] = (lse[on] ** 2).sum() / n
    return dict(ids=ids, weights=w, lse=lse, p=p, counts=counts, n=n, prob_sum=prob, loss=loss)


def gate_grad(g, k, renorm, d_weights, d_loss):
    """Gradient of sum(d_weights * weights) + sum(d_loss * loss) with respect to the logits, the counts
    constant, and (second) the sum of the magnitudes of its terms, the scale of its rounding."""
    T, E = g["p"].shape
    dl, mag = np.zeros((T, E)), np.zeros((T, E))
    n = max(g["n"], 1)
    c = np.zeros(E) if d_loss is None else d_loss[0] * E * g["counts"] / (k * n) / n
    cz = 0.0 if d_loss is None else 2.0 * d_loss[1] / n
    for t in range(T):
        if g["lse"][t] == -np.inf:
            continue
        p, q = g["p"][t], c.copy()
        on = g["ids"][t] >= 0
        sel, w = g["ids"][t][on], g["weights"][t][on]
        dw = np.zeros(sel.size) if d_weights is None else np.asarray(d_weights, np.float64)[t][on]
        if not renorm:
            q[sel] += dw
        dl[t] = p * (q - (p * q).sum() + cz * g["lse"][t])
        mag[t] = p * (np.abs(q) + (p * np.abs(q)).sum() + abs(cz * g["lse"][t]))
        if renorm:
            dl[t][sel] += w * (dw - (w * dw).sum())
            mag[t][sel] += w * (np.abs(dw) + (w * np.abs(dw)).sum())
    return dl, mag
