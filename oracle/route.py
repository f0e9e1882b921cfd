"""The router and the gradient of its logits in float64.  TEST INFRASTRUCTURE.

The pages start at the router's top-K output; the rule here is the library's own
(moonep.h, moonep_route). Experts are ranked by s + bias (by the logit where there is no
bias), groups first, ties to the lower id, masked experts last.
"""
from __future__ import annotations

import numpy as np


def _effective(logits, bias):
    """Logits that count: -inf where the bias is -inf, NaN where it is NaN."""
    l = np.array(logits, dtype=np.float64)
    if bias is not None:
        b = np.broadcast_to(np.asarray(bias, dtype=np.float64), l.shape)
        l = np.where(b == -np.inf, -np.inf, np.where(np.isnan(b), np.nan, l))
    return l


def _scores(l, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    m = np.max(np.where(np.isnan(l), -np.inf, l))
    with np.errstate(invalid="ignore"):
        ex = np.where(l == -np.inf, 0.0, np.exp(l - m))
        return ex / ex.sum() if ex.sum() != 0 else ex


def route(logits, bias, K, score="softmax", groups=1, top_groups=1, group_top=1, renorm=True,
          scale=1.0):
    """(topk_idx int32 [N, K], gates float64 [N, K])."""
    N, E = np.shape(logits)
    ids = np.zeros((N, K), dtype=np.int32)
    gates = np.zeros((N, K))
    per = E // groups
    for g in range(N):
        l = _effective(np.asarray(logits)[g], bias)
        s = _scores(l, score)
        masked = l == -np.inf
        total = s if bias is None else s + np.asarray(bias, dtype=np.float64)
        key = np.where(masked, -np.inf, l if bias is None else total)
        key = np.where(np.isnan(key), -np.inf, key)
        if groups > 1:
            worth = np.full(groups, -np.inf)
            for j in range(groups):
                mem = slice(j * per, (j + 1) * per)
                if group_top == 1:
                    worth[j] = key[mem].max()
                else:
                    # unmasked members by s + bias, the best one or two of them
                    live = sorted((v for v, mk in zip(total[mem], masked[mem])
                                   if not mk and not np.isnan(v)), reverse=True)[:2]
                    if live:
                        worth[j] = sum(live)
            stay = sorted(range(groups), key=lambda j: (-worth[j], j))[:top_groups]
            key = np.array([key[e] if e // per in stay else -np.inf for e in range(E)])
        order = sorted(range(E), key=lambda e: (-key[e], e))[:K]
        ids[g] = order
        live = [e for e in order if key[e] != -np.inf]
        if np.isnan(l).any() or (score == "softmax" and np.isposinf(l).any()):
            gates[g] = np.nan
            continue
        if renorm and live:
            # log-scores, so that the ratio survives scores that underflow
            if score == "softmax":
                ls = l[live]
            else:
                ls = np.where(l[live] < 0, l[live] - np.log1p(np.exp(np.minimum(l[live], 0))),
                              -np.log1p(np.exp(-np.maximum(l[live], 0))))
            w = np.exp(ls - ls.max())
            val = dict(zip(live, w / w.sum()))
        else:
            val = {e: s[e] for e in live}
        gates[g] = [scale * val.get(e, 0.0) for e in order]
    return ids, gates


def route_backward(logits, bias, topk_idx, gates, dgates, score="softmax", renorm=True, scale=1.0):
    """dlogits float64 [N, E], the formula of moonep_route_backward."""
    N, E = np.shape(logits)
    out = np.zeros((N, E))
    for g in range(N):
        l = _effective(np.asarray(logits)[g], bias)
        ga = np.asarray(gates, dtype=np.float64)[g]
        live = [k for k in range(len(ga)) if ga[k] != 0 and 0 <= topk_idx[g][k] < E]
        dg = np.asarray(dgates, dtype=np.float64)[g]
        mean = sum(ga[k] * dg[k] for k in live)
        if score == "softmax" and not renorm:
            out[g] = -_scores(l, score) * mean
        for k in live:
            v = ga[k] * (dg[k] - mean / scale if renorm else dg[k])
            if score == "sigmoid":
                with np.errstate(over="ignore"):
                    v *= 1.0 / (1.0 + np.exp(l[topk_idx[g][k]]))
            out[g, topk_idx[g][k]] += v
    return out
