"""fp64 reference of the token scoring and top-logit distillation operators -- TEST
INFRASTRUCTURE ONLY.

Definitions (x a row of logits, c = 1 / temperature, m = max x, S = sum_v exp(c (x_v - m))):
    logp_v  = c (x_v - m) - ln S           entropy = - sum_v p_v logp_v, p_v = exp(logp_v)
    top k   = the k largest x, the lowest id first among equal ones; NaN never
    d logp_i / dx_v = c ([v = i] - p_v)    d entropy / dx_v = - c p_v (logp_v + entropy)
    KL      = sum over listed v of T_v (ln T_v - logp_v) + P_R (ln P_R - ln q_R), T_v = sum over i with
              id_i = v of P_i (an id's entries are one class), q_R = sum of p outside the ids
    dKL/dx_v = c (p_v P - T_v - [v not listed] P_R p_v / q_R), P = sum_i P_i + P_R
A row with every logit at -inf: logp -inf, entropy 0, divergence 0, zero gradients."""
from __future__ import annotations

import numpy as np


def log_softmax(x, c=1.0):
    """Row log-probabilities, (m, ln S) and which rows are empty."""
    x = np.asarray(x, dtype=np.float64)
    m = x.max(axis=1)
    empty = m == -np.inf
    t = (x - np.where(empty, 0.0, m)[:, None]) * c
    with np.errstate(divide="ignore"):
        ls = np.log(np.exp(t).sum(axis=1))
    return np.where(empty[:, None], -np.inf, t - np.where(empty, 0.0, ls)[:, None]), m, ls, empty


def _plogp(lp):
    p = np.exp(lp)
    return p, np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0)


def score(x, ids, pred, c=1.0, k=0):
    """logp [N] (0 where pred < 0), (m, ln S) [N, 2], entropy [N], top ids and log-probabilities
    [N, k]; pred[t]: the row whose logits predict token t."""
    x = np.asarray(x, dtype=np.float64)
    lp, m, ls, empty = log_softmax(x, c)
    entropy = -_plogp(lp)[1].sum(axis=1)
    pred = np.asarray(pred)
    r = np.maximum(pred, 0)
    logp = np.where(pred < 0, 0.0, lp[r, np.asarray(ids)])
    top = np.argsort(np.where(np.isnan(x), np.inf, -x), axis=1, kind="stable")[:, :k]
    return logp, np.stack([m, ls], axis=1), entropy, top, np.take_along_axis(lp, top, axis=1)


def score_bwd(x, ids, pred, g_logp, g_entropy, c=1.0):
    x = np.asarray(x, dtype=np.float64)
    lp, _, _, empty = log_softmax(x, c)
    p, plp = _plogp(lp)
    H = -plp.sum(axis=1)
    d = np.zeros_like(x)
    if g_entropy is not None:
        d -= np.asarray(g_entropy, dtype=np.float64)[:, None] * (plp + p * H[:, None])
    if g_logp is not None:
        for t, r in enumerate(np.asarray(pred)):
            if r < 0 or r >= len(x):
                continue
            d[r] -= float(g_logp[t]) * p[r]
            d[r, ids[t]] += float(g_logp[t])
    d[empty] = 0.0
    return d * c


def distill(x, t_ids, t_val, w=None, c=1.0, tail=False, grad_scale=1.0):
    """KL [N] (without weights), loss, dx [N, V]."""
    x = np.asarray(x, dtype=np.float64)
    N, V = x.shape
    lp, _, _, empty = log_softmax(x, c)
    q = np.exp(lp)
    w = np.ones(N) if w is None else np.asarray(w, dtype=np.float64)
    kl, d = np.zeros(N), np.zeros_like(x)
    for r in range(N):
        live = (t_ids[r] >= 0) & (t_ids[r] < V) & (t_val[r] != -np.inf)
        if w[r] == 0 or empty[r] or (not tail and not live.any()):
            continue
        at, z = t_ids[r][live], t_val[r][live].astype(np.float64)
        lnP = z if tail else log_softmax(z[None], c)[0][0]
        P = np.exp(lnP)
        at, cls = np.unique(at, return_inverse=True)
        P = np.bincount(cls, weights=P, minlength=len(at))
        rest = max(0.0, 1.0 - P.sum()) if tail else 0.0
        out = np.ones(V, dtype=bool)
        out[at] = False
        qR = q[r][out].sum()
        if qR == 0:
            rest = 0.0
        with np.errstate(invalid="ignore"):
            kl[r] = np.where(P > 0, P * (np.log(np.where(P > 0, P, 1.0)) - lp[r, at]), 0.0).sum()
        d[r] = q[r] * (P.sum() + rest)
        d[r, at] -= P
        if rest > 0:
            kl[r] += rest * (np.log(rest) - np.log(qR))
            d[r][out] -= rest * q[r][out] / qR
        d[r] *= w[r] * c * grad_scale
    return kl, float((w * kl).sum()), d
