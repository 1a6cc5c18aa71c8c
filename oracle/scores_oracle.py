"""Plain float64 reference of a head's scores (TEST INFRASTRUCTURE ONLY): the
log-probabilities of given tokens, the entropy, the best words, and the
gradient of a loss on log-probabilities and entropy.  Written from the
definitions, a row at a time; shares no code with the HIP library.
"""

from __future__ import annotations

import numpy as np

__all__ = ["scores", "scores_grad"]


def _row(z, tau):
    """(ln p, p) of one row; NaN throughout where the row has no distribution."""
    with np.errstate(all="ignore"):
        top = z.max()
        if not np.isfinite(top) or np.isnan(z).any():
            return np.full(z.shape, np.nan), np.full(z.shape, np.nan)
        t = tau * (z - top)
        lp = t - np.log(np.exp(t).sum())
        return lp, np.exp(lp)


def _live(tokens, V):
    return tokens is None or any(0 <= y < V for y in tokens)


def scores(z, tokens, n, tau=1.0):
    """(logp [T, m], entropy [T], ids [T, n], top [T, n])."""
    z = np.asarray(z, np.float64)
    T, V = z.shape
    m = 0 if tokens is None else tokens.shape[1]
    logp, entropy = np.zeros((T, m)), np.zeros(T)
    ids, top = np.full((T, n), -1), np.full((T, n), -np.inf)
    for i in range(T):
        row = None if tokens is None else tokens[i]
        if not _live(row, V):
            continue
        lp, p = _row(z[i], tau)
        for j in range(m):
            if 0 <= row[j] < V:
                logp[i, j] = lp[row[j]]
        entropy[i] = -(p[p > 0] * lp[p > 0]).sum() if not np.isnan(p).any() else np.nan
        if np.isnan(p).any():
            top[i] = np.nan
            continue
        for j, v in enumerate(np.argsort(-z[i], kind="stable")[:n]):
            if z[i, v] > -np.inf:
                ids[i, j], top[i, j] = v, lp[v]
    return logp, entropy, ids, top


def scores_grad(z, tokens, dlogp, dentropy, tau=1.0):
    """Gradient of sum(dlogp logp) + sum(dentropy entropy) in z."""
    z = np.asarray(z, np.float64)
    T, V = z.shape
    out = np.zeros(z.shape)
    for i in range(T):
        row = None if tokens is None else tokens[i]
        if not _live(row, V):
            continue
        use = [] if row is None else [j for j in range(len(row)) if 0 <= row[j] < V]
        gh = 0.0 if dentropy is None else float(dentropy[i])
        if gh == 0 and all(dlogp[i, j] == 0 for j in use):
            continue
        lp, p = _row(z[i], tau)
        total = sum(float(dlogp[i, j]) for j in use)
        plp = np.where(p > 0, p * np.where(p > 0, lp, 0.0), p)
        out[i] = -total * p - gh * (plp - p * plp.sum())
        for j in use:
            out[i, row[j]] += float(dlogp[i, j])
    return out * tau
