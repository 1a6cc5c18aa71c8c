"""Plain float64 reference of the fine-tuning step around the adapted linear
(TEST INFRASTRUCTURE ONLY): label log-probabilities under a head's logits,
the preference loss, the clipped policy loss with a KL term, and momentum with
an orthogonalised update.  Written from the definitions, one sequence, token
or matrix at a time; shares no code with the HIP library.
"""

from __future__ import annotations

import numpy as np

__all__ = ["label_logprobs", "label_logprobs_grad", "preference", "policy", "orthogonalised", "muon"]


def _softmax(z, tau):
    with np.errstate(invalid="ignore"):
        t = tau * (z - np.max(z))
        e = np.exp(t)
        return t, e, e.sum()


def label_logprobs(z, labels, tau=1.0):
    """logp[t] = tau z_y - ln sum_v exp(tau z_v); 0 where y is outside [0, V)."""
    z = np.asarray(z, np.float64)
    out = np.zeros(z.shape[0])
    for i, y in enumerate(labels):
        if 0 <= y < z.shape[1]:
            t, _, s = _softmax(z[i], tau)
            out[i] = t[y] - np.log(s)
    return out


def label_logprobs_grad(z, labels, dlogp, tau=1.0):
    """dlogp[t] tau ([v = y] - p_v), 0 where the token does not count or dlogp is 0."""
    z = np.asarray(z, np.float64)
    out = np.zeros(z.shape)
    for i, y in enumerate(labels):
        if 0 <= y < z.shape[1] and dlogp[i] != 0:
            _, e, s = _softmax(z[i], tau)
            out[i] = -e / s
            out[i, y] += 1.0
            out[i] *= dlogp[i] * tau
    return out


def preference(logp, labels, vocab, cu, beta, ref=None, kind="sigmoid", average=False, smoothing=0.0, margin=0.0,
               weight=None):
    """(loss [P], reward [2P], dlogp [T]): pairs (p, P + p) of sequences cu[s]..cu[s+1]-1."""
    P = (len(cu) - 1) // 2
    logp = np.asarray(logp, np.float64)
    gain, count = np.zeros(2 * P), np.ones(2 * P)
    for s in range(2 * P):
        inside = [t for t in range(cu[s], cu[s + 1]) if 0 <= labels[t] < vocab]
        gain[s] = sum(logp[t] - (ref[t] if ref is not None else 0.0) for t in inside)
        if average:
            count[s] = max(1, len(inside))
    gain /= count
    loss, dlogp = np.zeros(P), np.zeros(len(logp))
    for p in range(P):
        h = beta * (gain[p] - gain[P + p]) - margin
        if kind == "sigmoid":
            loss[p] = (1 - smoothing) * np.logaddexp(0, -h) + smoothing * np.logaddexp(0, h)
            dh = 1 / (1 + np.exp(-h)) - (1 - smoothing)
        elif kind == "hinge":
            loss[p], dh = max(0.0, 1 - h), -1.0 if h < 1 else 0.0
        else:
            loss[p], dh = ((h - 0.5) / beta) ** 2, 2 * (h - 0.5) / beta ** 2
        w = 1.0 if weight is None else float(weight[p])
        for s, sign in ((p, 1.0), (P + p, -1.0)):
            for t in range(cu[s], cu[s + 1]):
                if 0 <= labels[t] < vocab:
                    dlogp[t] = sign * w * dh * beta / count[s]
    return loss, beta * gain, dlogp


def policy(logp, labels, vocab, adv, old=None, ref=None, weight=None, low=0.2, high=0.2, kl_coef=0.0):
    """(loss [T], kl [T], dlogp [T]) from label log-probabilities."""
    T = len(logp)
    loss, kl, g = np.zeros(T), np.zeros(T), np.zeros(T)
    for t in range(T):
        if not 0 <= labels[t] < vocab:
            continue
        r = np.exp(logp[t] - old[t]) if old is not None else 1.0
        x, y = r * adv[t], min(max(r, 1 - low), 1 + high) * adv[t]
        loss[t] = -min(x, y)
        g[t] = -x if x <= y else 0.0
        if ref is not None:
            d = ref[t] - logp[t]
            kl[t] = np.exp(d) - d - 1
            loss[t] += kl_coef * kl[t]
            g[t] += kl_coef * (1 - np.exp(d))
        if weight is not None:
            g[t] *= weight[t]
    return loss, kl, g


USUAL = (3.4445, -4.7750, 2.0315)


def orthogonalised(u, coef, eps=1e-7):
    """Newton-Schulz steps on one matrix, in its own shape."""
    x = np.asarray(u, np.float64)
    x = x / (np.sqrt((x * x).sum()) + eps)
    for a, b, c in coef:
        if x.shape[0] <= x.shape[1]:
            g = x @ x.T
            x = a * x + b * (g @ x) + c * (g @ (g @ x))
        else:
            g = x.T @ x
            x = a * x + b * (x @ g) + c * ((x @ g) @ g)
    return x


def muon(W, g, m, lr, momentum=0.95, nesterov=True, wd=0.0, coef=(USUAL,) * 5, scale=None, eps=1e-7):
    """(W, m) after one step on one matrix."""
    W, g, m = (np.asarray(v, np.float64) for v in (W, g, m))
    m = momentum * m + g
    u = g + momentum * m if nesterov else m
    if scale is None:
        scale = max(1.0, W.shape[0] / W.shape[1]) ** 0.5
    return (1 - lr * wd) * W - lr * scale * orthogonalised(u, coef, eps), m
