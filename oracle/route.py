"""The expert router, its balance loss and gradients, and the sum of the slots, in fp64 (test infrastructure)."""

import numpy as np


def route(logits, S, normalise, coef, valid=None):
    """dict of ids [N, S] (-1: none left), weights, counts [E + 1], psum [E], loss, p [N, E]; row by row."""
    l = np.asarray(logits, dtype=np.float64)
    N, E = l.shape
    ids, weights = np.full((N, S), -1, np.int32), np.zeros((N, S))
    p, counts = np.zeros((N, E)), np.zeros(E + 1, np.int64)
    for t in range(N):
        if valid is not None and not valid[t]:
            continue
        able = [e for e in range(E) if l[t, e] > -np.inf]   # neither -inf nor NaN
        if not able:
            continue
        counts[E] += 1
        chosen = sorted(able, key=lambda e: (-l[t, e], e))[:S]
        with np.errstate(invalid="ignore", over="ignore"):
            ex = np.exp(l[t] - l[t, chosen[0]])
            p[t] = ex / ex.sum()
        ids[t, :len(chosen)] = chosen
        w = p[t, chosen]
        weights[t, :len(chosen)] = w / w.sum() if normalise else w
        if normalise and np.isnan(p[t]).any():
            weights[t, :len(chosen)] = np.nan
        for e in chosen:
            counts[e] += 1
    psum = p.sum(0)
    return dict(ids=ids, weights=weights, counts=counts, psum=psum, p=p, loss=balance_loss(counts, psum, S, coef))


def balance_loss(counts, psum, S, coef):
    E, T = len(psum), counts[-1]
    if T == 0:
        return 0.0
    f = counts[:E].astype(np.float64) * E / (S * T)
    return coef * float((f * np.asarray(psum, dtype=np.float64)).sum()) / T


def route_backward(logits, r, normalise, coef, dweights=None, dloss=None):
    """dlogits of sum(dweights * weights) + dloss * loss with f_e held fixed; r = route(...)."""
    l = np.asarray(logits, dtype=np.float64)
    N, E = l.shape
    S = r["ids"].shape[1]
    T = r["counts"][E]
    out = np.zeros((N, E))
    f = r["counts"][:E].astype(np.float64) * E / (S * T) if T else np.zeros(E)
    for t in range(N):
        p = r["p"][t]
        if not p.any():
            continue
        dp = dloss * coef * f / T if dloss is not None else np.zeros(E)
        dp = dp.copy()
        if dweights is not None:
            k = r["ids"][t] >= 0
            ids, dw, w = r["ids"][t][k], np.asarray(dweights[t], dtype=np.float64)[k], r["weights"][t][k]
            dp[ids] += (dw - (dw * w).sum()) / p[ids].sum() if normalise else dw
        out[t] = p * (dp - (p * dp).sum())
    return out


def combine(y, w=None):
    """Sum over the slots, a slot of weight 0 left out whatever it holds."""
    y = np.asarray(y, dtype=np.float64)
    if w is None:
        return y.sum(1)
    w = np.asarray(w, dtype=np.float64)[:, :, None]
    return (np.where(w == 0, 0, y) * w).sum(1)
