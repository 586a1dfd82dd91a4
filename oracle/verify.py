"""fp64 reference of the verification of drafted tokens -- TEST INFRASTRUCTURE ONLY.

Row r of a cursor leads to the draft in row r + 1.  With p = softmax(c x_r), q = softmax(cq y_r):
    a = min(1, p(id) / q(id)), 0 where p(id) is 0 in fp64 (q = 1 without draft logits), accepted iff u < a;
    next token after the first rejected one: argmax max(0, p - q) / noise (without draft logits p
    with the rejected id left out), p / noise where nothing is left or all were accepted; the lowest
    id among equal ones.
Greedy (u, noise None): accepted iff id is the largest logit's lowest id.  A row with a NaN has its draft
rejected and gives no token."""
from __future__ import annotations

import numpy as np

from .token_score import log_softmax


def _first(score):
    score = np.where(np.isnan(score), 0.0, score)
    return int(np.argmax(score)) if score.max() > 0 else -1


def _largest(x):
    """Lowest id of the largest logit; -1 where none is above -inf or one is NaN."""
    return -1 if np.isnan(x).any() or not x.max(initial=-np.inf) > -np.inf else int(np.argmax(x))


def verify(x, rows, ids, y=None, u=None, noise=None, c=1.0, cq=1.0):
    """n_accept, next_id, next_logp [cursors], accept_p [rows]; rows: rows of each cursor."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        lp = log_softmax(x, c)[0] if len(x) else x
        lq = None if y is None else log_softmax(y, cq)[0]
    n_accept, next_id, next_logp, accept = [], [], [], np.zeros(len(x))
    greedy = u is None
    r0 = 0
    for i, n in enumerate(rows):
        if n == 0:
            n_accept.append(0), next_id.append(-1), next_logp.append(-np.inf)
            continue
        r, w = r0, None
        while r + 1 < r0 + n:
            t = int(ids[r + 1])
            if t < 0 or t >= x.shape[1]:
                a, t = 0.0, -1
            elif greedy:
                a = float(_largest(x[r]) == t)
            else:
                with np.errstate(invalid="ignore", over="ignore"):
                    a = 0.0 if np.exp(lp[r, t]) == 0 else float(np.exp(min(0.0, lp[r, t] - (lq[r, t] if lq is not None else 0.0))))
                if np.isnan(lp[r, t]) or (lq is not None and np.isnan(lq[r, t])):
                    a = 0.0
            accept[r + 1] = a
            if a > 0 if greedy else u[r + 1] < a:
                r += 1
                continue
            if not greedy:
                p = np.exp(lp[r])
                if lq is not None:
                    with np.errstate(invalid="ignore"):
                        w = np.maximum(p - np.exp(lq[r]), 0.0)
                else:
                    w = p.copy()
                    if t >= 0:
                        w[t] = 0.0
            break
        p = np.exp(lp[r])
        if greedy:
            best = _largest(x[r])
        else:
            best = -1 if w is None else _first(w / noise[i])
            if best < 0:
                best = _first(p / noise[i])
        n_accept.append(r - r0), next_id.append(best), next_logp.append(lp[r, best] if best >= 0 else -np.inf)
        r0 += n
    return np.array(n_accept), np.array(next_id), np.array(next_logp), accept
